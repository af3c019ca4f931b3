// list_norms.cu -- the norms of every tensor of a list, of groups of tensors
// and of all of them (p = 1, 2, infinity), tensors of mixed types.
//
//  1. chunk_sums_kernel: one block per chunk (4096 to 65536 elements, never
//     across two tensors) reads it once and leaves one binary64 partial: for
//     p = 2 the squares in double-float pairs (NormAcc of reduce.cuh; exact
//     squares for 16-bit elements), for p = 1 the magnitudes in the same
//     pairs, for infinity the largest magnitude by its bits (a NaN's are the
//     largest, so it stays).  A chunk whose squares leave the binary32 range
//     is read again scaled by a power of two, which is exact.
//  2. tensor_sums_kernel: the partials of each tensor in a fixed order, times
//     |scale|^p.
//  3. norms_kernel: the sums of each group's tensors, and of all; roots,
//     coefficients.
//
// No atomics: the result is bit-identical from run to run.
#include "common.cuh"
#include "grad_list.cuh"
#include "kernels.h"

namespace zs {

// ------------------------------------------------------------ 1: chunks
// What a thread gathers of its elements: the sums, and in `bits` the elements'
// bits or'ed (p = 2: whether any is not zero) or the largest magnitude's
// (infinity).
template <int P>
struct Gather {
  NormAcc acc;
  uint32_t bits = 0u;

  // Magnitudes are added as NormAcc adds squares that leave no residual.
  __device__ __forceinline__ void add_abs(float x0, float x1) {
    const unsigned long long p = f2_pack(fabsf(x0), fabsf(x1));
    const unsigned long long s = f2_add(acc.h, p);
    const unsigned long long bp = f2_sub(s, acc.h);
    const unsigned long long t = f2_add(f2_sub(acc.h, f2_sub(s, bp)), f2_sub(p, bp));
    acc.h = s;
    acc.l = f2_add(acc.l, t);
  }
  template <bool EXACT>
  __device__ __forceinline__ void pair(float x0, float x1) {
    if (P == ZERO_NORM_1)
      add_abs(x0, x1);
    else if (EXACT)
      acc.add2_exact(f2_pack(x0, x1));
    else
      acc.add2(x0, x1);
  }
  // 8 elements of 16 bits
  template <int DT>
  __device__ __forceinline__ void vec16(const uint4& w) {
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
    if (P == ZERO_NORM_INF) {
#pragma unroll
      for (int j = 0; j < 4; ++j) bits = __vmaxu2(bits, ws[j] & 0x7fff7fffu);
      return;
    }
    if (P == ZERO_NORM_2) bits |= (w.x | w.y) | (w.z | w.w);
#pragma unroll
    for (int j = 0; j < 4; ++j) pair<true>(half_bits_to_f32<DT>(ws[j] & 0xffffu), half_bits_to_f32<DT>(ws[j] >> 16));
  }
  __device__ __forceinline__ void vec32(const float (&x)[8]) {
    if (P == ZERO_NORM_INF) {
#pragma unroll
      for (int j = 0; j < 8; ++j) bits = max(bits, __float_as_uint(x[j]) & 0x7fffffffu);
      return;
    }
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      if (P == ZERO_NORM_2) bits |= __float_as_uint(x[j]) | __float_as_uint(x[j + 1]);
      pair<false>(x[j], x[j + 1]);
    }
  }
  // one element of the head or tail
  template <int DT>
  __device__ __forceinline__ void one(const void* p, int e) {
    if (DT == ZERO_F32) {
      const uint32_t b = __float_as_uint(load_elem<DT>(p, e));
      if (P == ZERO_NORM_INF) {
        bits = max(bits, b & 0x7fffffffu);
      } else {
        bits |= b;
        pair<false>(__uint_as_float(b), 0.0f);
      }
    } else {
      const uint32_t h = __ldg(static_cast<const unsigned short*>(p) + e);
      if (P == ZERO_NORM_INF) {
        bits = __vmaxu2(bits, h & 0x7fffu);
      } else {
        bits |= h;
        pair<true>(half_bits_to_f32<DT>(h), 0.0f);
      }
    }
  }
  // the largest magnitude's binary32 bits (infinity)
  template <int DT>
  __device__ __forceinline__ uint32_t top() const {
    if (DT == ZERO_F32) return bits;
    return max(__float_as_uint(half_bits_to_f32<DT>(bits & 0xffffu)),
               __float_as_uint(half_bits_to_f32<DT>(bits >> 16)));
  }
  // whether any element is not zero (p = 2)
  template <int DT>
  __device__ __forceinline__ bool any() const {
    return (bits & (DT == ZERO_F32 ? 0x7fffffffu : 0x7fff7fffu)) != 0u;
  }
};

// Every thread's result.
__device__ __forceinline__ uint32_t block_max(uint32_t m, uint32_t* red) {
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kGradThreads / 32; ++w) m = max(m, red[w]);
  __syncthreads();
  return m;
}

// A chunk again, its elements scaled so that the largest lies in [1, 2): the
// sum of squares (magnitudes) of any finite elements.  An element whose
// square loses bits then is below 2^-62 of the largest.  Thread 0's result.
template <int P, int DT>
__device__ __noinline__ double scaled_sum(const void* p, int len, float2* red) {
  uint32_t m = 0u;
  for (int e = threadIdx.x; e < len; e += kGradThreads)
    m = max(m, __float_as_uint(load_elem<DT>(p, e)) & 0x7fffffffu);
  m = block_max(m, reinterpret_cast<uint32_t*>(red));
  if (m >= 0x7f800000u) return static_cast<double>(__uint_as_float(m));  // infinite, or a NaN
  if (m == 0u) return 0.0;
  const int e2 = ilogbf(__uint_as_float(m));
  Gather<P> g;
  for (int e = threadIdx.x; e < len; e += kGradThreads) g.template pair<false>(scalbnf(load_elem<DT>(p, e), -e2), 0.0f);
  return scalbn(block_sum_norm<kGradThreads>(g.acc, red), P == ZERO_NORM_2 ? 2 * e2 : e2);
}

// The partial of elements [0, len) at p, in thread 0.
template <int P, int DT>
__device__ __forceinline__ double chunk_sum(const void* p, int len, float2* red) {
  constexpr int es = SrcTraits<DT>::esize;
  constexpr int kAhead = (DT == ZERO_F32) ? 4 : 8;  // vectors in flight per thread
  const Run r = vector_run<es>(p, len);
  const char* body = static_cast<const char*>(p) + es * r.head;
  Gather<P> g;
  for (int v0 = threadIdx.x; v0 < r.vecs; v0 += kAhead * kGradThreads) {
    if (DT == ZERO_F32) {
      float x[kAhead][8];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int v = v0 + u * kGradThreads;
        if (v < r.vecs && ZS_CHECK(aligned(body + 32 * v, 32) && r.head + 8 * v + 8 <= len, 70, v)) {
          ld8_ro(reinterpret_cast<const float*>(body) + 8 * v, x[u]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[u][i] = 0.0f;
        }
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) g.vec32(x[u]);
    } else {
      uint4 w[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int v = v0 + u * kGradThreads;
        w[u] = make_uint4(0u, 0u, 0u, 0u);
        if (v < r.vecs && ZS_CHECK(aligned(body + 16 * v, 16) && r.head + 8 * v + 8 <= len, 71, v))
          w[u] = ld16_ro(body + 16 * v);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) g.template vec16<DT>(w[u]);
    }
  }
  const int e = ragged_element(r, len);
  if (e >= 0 && ZS_CHECK(e < len, 72, e)) g.template one<DT>(p, e);
  if (P == ZERO_NORM_INF)
    return static_cast<double>(__uint_as_float(block_max(g.template top<DT>(), reinterpret_cast<uint32_t*>(red))));
  const double sum = block_sum_norm<kGradThreads>(g.acc, red);
  // Squares below 2^-126 have lost bits: at most 2^-150 each, 2^-134 of a
  // chunk, so a sum of 2^-80 and more is right to 2^-54.  Magnitudes lose none.
  const bool fits = sum < static_cast<double>(INFINITY) && (P == ZERO_NORM_1 || sum >= 0x1p-80);
  if (__syncthreads_and(threadIdx.x != 0 || fits)) return sum;
  if (P == ZERO_NORM_2 && !__syncthreads_or(g.template any<DT>())) return 0.0;
  return scaled_sum<P, DT>(p, len, red);
}

template <int P>
__global__ void __launch_bounds__(kGradThreads)
    chunk_sums_kernel(const zero_grad_entry* __restrict__ entries, int n, const int32_t* __restrict__ first, int chunk,
                      double* __restrict__ partials) {
  __shared__ float2 red[kGradThreads / 32];
  const GradChunk c = grad_chunk(entries, first, n, chunk, blockIdx.x);
  const zero_grad_entry& t = entries[c.tensor];
  if (!ZS_CHECK(c.len > 0 && c.k >= 0 && c.k + c.len <= t.numel, 73, blockIdx.x)) return;
  const char* src = static_cast<const char*>(t.src);
  double sum = 0.0;
  if (src != nullptr) {
    if (t.src_dtype == ZERO_F32)
      sum = chunk_sum<P, ZERO_F32>(src + 4 * c.k, c.len, red);
    else if (t.src_dtype == ZERO_BF16)
      sum = chunk_sum<P, ZERO_BF16>(src + 2 * c.k, c.len, red);
    else
      sum = chunk_sum<P, ZERO_F16>(src + 2 * c.k, c.len, red);
  }
  if (threadIdx.x == 0) partials[blockIdx.x] = sum;
}

// ----------------------------------------------------------- 2: tensors
// The two ways of joining: sums, and the largest with NaN above all.
template <int P>
__device__ __forceinline__ double join(double a, double b) {
  if (P != ZERO_NORM_INF) return a + b;
  return (a > b || a != a) ? a : b;
}

template <int P>
__device__ __forceinline__ double warp_join(double x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x = join<P>(x, __shfl_down_sync(0xffffffffu, x, off));
  return x;
}

// Thread 0's result; every thread of the block must call it.
template <int P, int THREADS>
__device__ __forceinline__ double block_join(double x, double* red) {
  x = warp_join<P>(x);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  double r = red[0];
  if (threadIdx.x == 0)
    for (int w = 1; w < THREADS / 32; ++w) r = join<P>(r, red[w]);
  __syncthreads();
  return r;
}

// load(at), load(at + step), ... below count, eight in flight.
template <int P, class Load>
__device__ __forceinline__ double strided(int at, int count, int step, const Load& load) {
  double acc = 0.0;
  for (int64_t i = at; i < count; i += 8 * step) {
    double v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = i + u * step < count ? load(static_cast<int>(i + u * step)) : 0.0;
#pragma unroll
    for (int u = 0; u < 8; ++u) acc = join<P>(acc, v[u]);
  }
  return acc;
}

// Partials up to which one warp adds a tensor's; above, the block does.
constexpr int kWarpPartials = 2048;

template <int P>
__global__ void __launch_bounds__(kGradThreads)
    tensor_sums_kernel(const double* __restrict__ partials, const int32_t* __restrict__ first, int n, float scale,
                       const float* __restrict__ dscale, double* __restrict__ sums) {
  __shared__ double red[kGradThreads / 32];
  const double s = fabs(static_cast<double>(dscale != nullptr ? *dscale : scale));
  const double factor = P == ZERO_NORM_2 ? s * s : s;
  const int base = blockIdx.x * (kGradThreads / 32);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int mine = base + warp;
  if (mine < n) {
    const int lo = __ldg(first + mine), count = __ldg(first + mine + 1) - lo;
    if (count <= kWarpPartials) {
      const double x = warp_join<P>(strided<P>(lane, count, 32, [&](int i) { return __ldg(partials + lo + i); }));
      if (lane == 0) sums[mine] = x * factor;
    }
  }
  for (int i = base; i < min(base + kGradThreads / 32, n); ++i) {
    const int lo = __ldg(first + i), count = __ldg(first + i + 1) - lo;
    if (count <= kWarpPartials) continue;
    const double x = block_join<P, kGradThreads>(
        strided<P>(threadIdx.x, count, kGradThreads, [&](int j) { return __ldg(partials + lo + j); }), red);
    if (threadIdx.x == 0) sums[i] = x * factor;
  }
}

// ------------------------------------------------------ 3: groups and all
constexpr int kNormThreads = 1024;

struct NormsArgs {
  GradPlan plan;
  int n, n_groups;
  const double* sums;
  int n_parts;
  const double* max_norms;
  float* norms;
  zero_norm_result* results;
  int32_t* found;
};

template <int P>
__device__ __forceinline__ double root(double s) {
  return P == ZERO_NORM_2 ? __dsqrt_rn(s) : s;
}

// Tensor i's sum over the parts, in their order.
template <int P>
__device__ __forceinline__ double tensor_sum(const NormsArgs& a, int i) {
  double s = __ldg(a.sums + i);
  for (int r = 1; r < a.n_parts; ++r) s = join<P>(s, __ldg(a.sums + static_cast<int64_t>(r) * a.n + i));
  return s;
}

template <int P>
__device__ __forceinline__ void write_result(const NormsArgs& a, int g, double sum) {
  const double norm = root<P>(sum);
  zero_norm_result r;
  r.sqnorm = sum;
  r.norm = norm;
  r.clip_coef = 1.0f;
  r.finite = isfinite(norm) ? 1 : 0;
  if (g < a.n_groups) {
    const double q = __ddiv_rn(__ldg(a.max_norms + g), __dadd_rn(norm, 1e-6));
    if (q < 1.0) r.clip_coef = __double2float_rn(q);
  } else if (a.found != nullptr && !r.finite) {
    *a.found = 1;
  }
  a.results[g] = r;
  a.norms[a.n + g] = __double2float_rn(norm);
}

// Block 0: all tensors.  The others: a group each (WARPS == false), or 32
// groups, a warp each, where groups are small.
template <int P, bool WARPS>
__global__ void __launch_bounds__(kNormThreads) norms_kernel(const __grid_constant__ NormsArgs a) {
  __shared__ double red[kNormThreads / 32];
  if (blockIdx.x == 0) {
    const double s = block_join<P, kNormThreads>(
        strided<P>(threadIdx.x, a.n, kNormThreads, [&](int i) { return tensor_sum<P>(a, i); }), red);
    if (threadIdx.x == 0) write_result<P>(a, a.n_groups, s);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = WARPS ? (blockIdx.x - 1) * (kNormThreads / 32) + warp : blockIdx.x - 1;
  if (g >= a.n_groups) return;  // WARPS: a whole warp, and no barrier follows
  const int lo = __ldg(a.plan.group_first + g), count = __ldg(a.plan.group_first + g + 1) - lo;
  const auto member = [&](int j) {
    const int i = __ldg(a.plan.members + lo + j);
    const double s = tensor_sum<P>(a, i);
    a.norms[i] = __double2float_rn(root<P>(s));
    return s;
  };
  if (WARPS) {
    const double s = warp_join<P>(strided<P>(lane, count, 32, member));
    if (lane == 0) write_result<P>(a, g, s);
  } else {
    const double s = block_join<P, kNormThreads>(strided<P>(threadIdx.x, count, kNormThreads, member), red);
    if (threadIdx.x == 0) write_result<P>(a, g, s);
  }
}

// -------------------------------------------------------------- launches
template <int P>
static zero_status launch_sums_t(const GradListArgs& a, double* partials, double* sums, cudaStream_t st) {
  const GradPlan plan = plan_parts(a.plan, a.n, a.n_groups);
  if (a.n_chunks > 0) {
    chunk_sums_kernel<P><<<a.n_chunks, kGradThreads, 0, st>>>(a.entries, a.n, plan.first, a.chunk, partials);
    const zero_status s = check_launch("chunk_sums_kernel");
    if (s != ZERO_OK) return s;
  }
  tensor_sums_kernel<P><<<one_pass_blocks(a.n, kGradThreads / 32), kGradThreads, 0, st>>>(partials, plan.first, a.n,
                                                                                       a.scale, a.dscale, sums);
  return check_launch("tensor_sums_kernel");
}

template <int P>
static zero_status launch_norms_t(const NormsArgs& a, cudaStream_t st) {
  if (a.n / a.n_groups >= 256 || a.n_groups <= 64) {
    norms_kernel<P, false><<<1 + a.n_groups, kNormThreads, 0, st>>>(a);
  } else {
    norms_kernel<P, true><<<1 + one_pass_blocks(a.n_groups, kNormThreads / 32), kNormThreads, 0, st>>>(a);
  }
  return check_launch("norms_kernel");
}

ZS_DEBUG_UNIT(list_norms)

zero_status launch_list_sums(const GradListArgs& a, double* partials, double* sums, cudaStream_t st) {
  if (a.norm_type == ZERO_NORM_2) return launch_sums_t<ZERO_NORM_2>(a, partials, sums, st);
  if (a.norm_type == ZERO_NORM_1) return launch_sums_t<ZERO_NORM_1>(a, partials, sums, st);
  return launch_sums_t<ZERO_NORM_INF>(a, partials, sums, st);
}

zero_status launch_sums_norms(const GradListArgs& a, const double* sums, int n_parts, const double* max_norms,
                              float* norms, zero_norm_result* results, int32_t* found, cudaStream_t st) {
  const NormsArgs k{plan_parts(a.plan, a.n, a.n_groups), a.n, a.n_groups, sums, n_parts, max_norms, norms, results, found};
  if (a.norm_type == ZERO_NORM_2) return launch_norms_t<ZERO_NORM_2>(k, st);
  if (a.norm_type == ZERO_NORM_1) return launch_norms_t<ZERO_NORM_1>(k, st);
  return launch_norms_t<ZERO_NORM_INF>(k, st);
}

}  // namespace zs
