// list_norms.cu -- the norms of every tensor of a list, of groups of tensors
// and of all of them (p = 1, 2, infinity), tensors of mixed types.
//
//  1. chunk_sums_kernel: one block per wide chunk (4096 to 131072 elements,
//     never across two tensors) and one warp per narrow tensor read their
//     piece once and leave one binary64 partial: for p = 2 the squares in
//     double-float pairs (NormAcc of reduce.cuh; exact squares for 16-bit
//     elements), for p = 1 the magnitudes in the same pairs, for infinity the
//     largest magnitude by its bits (a NaN's are the largest, so it stays).
//     A piece whose squares leave the binary32 range is read again scaled by
//     a power of two, which is exact.
//  2. finish_kernel, one cluster or block: the partials of each tensor in a
//     fixed order, times |scale|^p; the norms of tensors, groups and all.  For
//     more than 1024 tensors or groups tensors_kernel and groups_kernel, over
//     all SMs.
//
// Bound by HBM from about 100 MB on: 1.63e9 fp16 elements, p = infinity, 454 us
// = 7.2 TB/s; 1.07e9 bf16, p = 2, 302 us = 7.1 TB/s (issue slots half busy, a
// third of the FMA pipe); 124e6 fp32, p = 1, 84 us = 5.9 TB/s, of which 72 are
// step 1; 20,000 ragged tensors of mixed types (3.1 GB) 457 us = 6.7 TB/s.
// Below, by latency: 1.3e6 fp32 elements 7.1 us, 5.4 without the results of
// groups and all.  A warp for every chunk of 16384 was slower (1.63e9: 549
// against 491 us: more places of memory read at once), one block of 256
// threads per chunk and tensor too (20,000 tensors: 565 us).
//
// No floating-point atomics: the result is bit-identical from run to run.
#include <cooperative_groups.h>

#include "common.cuh"
#include "grad_list.cuh"
#include "kernels.h"

namespace zs {

namespace cg = cooperative_groups;

// ------------------------------------------------------------ 1: chunks
// Threads of a block, vectors of 8 that a thread has in flight, and blocks on
// an SM (72 registers, of which p = 2 spills 4 bytes and infinity 20).
// Llama-7B's four layers in bf16, us: 304; with 8 blocks (64 registers, more
// spilled) 313, with 6 and 3 vectors 310, with blocks of 64 or 192 323 and 309.
constexpr int kSumThreads = 128, kAhead16 = 8, kAhead32 = 4, kSumBlocks = 7;

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
      const uint32_t b = __float_as_uint(elem_behind<DT>(p, e));
      if (P == ZERO_NORM_INF) {
        bits = max(bits, b & 0x7fffffffu);
      } else {
        bits |= b;
        pair<false>(__uint_as_float(b), 0.0f);
      }
    } else {
      const uint32_t h = bits_behind<DT>(p, e);
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

// A piece is summed by T threads: a block's, or one warp.
template <int T>
__device__ __forceinline__ int thread_of() {
  return T == 32 ? static_cast<int>(threadIdx.x & 31) : static_cast<int>(threadIdx.x);
}

// The T threads' sums in double-float, in a fixed order, rounded once to
// binary64: thread 0's result.
template <int T>
__device__ __forceinline__ double sum_norm(const NormAcc& acc, float2* red) {
  if (T != 32) return block_sum_norm<T>(acc, red);
  DF x = acc.value();
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
    x = df_add(x, DF{__shfl_down_sync(0xffffffffu, x.h, off), __shfl_down_sync(0xffffffffu, x.l, off)});
  return static_cast<double>(x.h) + static_cast<double>(x.l);
}

// Every thread's result.
template <int T>
__device__ __forceinline__ uint32_t max_of(uint32_t m, uint32_t* red) {
  m = __reduce_max_sync(0xffffffffu, m);
  if (T == 32) return m;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < T / 32; ++w) m = max(m, red[w]);
  __syncthreads();
  return m;
}
template <int T>
__device__ __forceinline__ bool any_of(bool x) {
  return T == 32 ? __any_sync(0xffffffffu, x) : __syncthreads_or(x) != 0;
}

// A piece again, its elements scaled so that the largest lies in [1, 2): the
// sum of squares (magnitudes) of any finite elements.  An element whose
// square loses bits then is below 2^-62 of the largest.  A thread adds its
// elements in pairs, as in the first pass: 512 of a chunk of 131072 for each
// lane, by which the error of the sum is bounded (a lane that takes all 1024
// was seen to be 9.3e-10 off, with elements made for that).  Thread 0's result.
template <int P, int DT, int T>
__device__ __noinline__ double scaled_sum(const void* p, int len, float2* red) {
  uint32_t m = 0u;
  for (int e = thread_of<T>(); e < len; e += T) m = max(m, __float_as_uint(elem_behind<DT>(p, e)) & 0x7fffffffu);
  m = max_of<T>(m, reinterpret_cast<uint32_t*>(red));
  if (m >= 0x7f800000u) return static_cast<double>(__uint_as_float(m));  // infinite, or a NaN
  if (m == 0u) return 0.0;
  const int e2 = ilogbf(__uint_as_float(m));
  Gather<P> g;
  for (int e = thread_of<T>(); e < len; e += 2 * T)
    g.template pair<false>(scalbnf(elem_behind<DT>(p, e), -e2),
                           e + T < len ? scalbnf(elem_behind<DT>(p, e + T), -e2) : 0.0f);
  return scalbn(sum_norm<T>(g.acc, red), P == ZERO_NORM_2 ? 2 * e2 : e2);
}

// N vectors of 8, T apart, from number v of `body` on, all loaded
// before the first is used; those from r.vecs on are left out unless FULL.
template <int P, int DT, int T, int N, bool FULL>
__device__ __forceinline__ void gather_vectors(const char* body, int v, const Run& r, int len, Gather<P>& g) {
  if (DT == ZERO_F32) {
    float x[N][8];
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const int k = v + T * u;
      if ((FULL || k < r.vecs) && ZS_CHECK(aligned(body + 32 * k, 32) && r.head + 8 * k + 8 <= len, 70, k)) {
        ld8_behind(reinterpret_cast<const float*>(body) + 8 * k, x[u]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[u][i] = 0.0f;
      }
    }
#pragma unroll
    for (int u = 0; u < N; ++u) g.vec32(x[u]);
  } else {
    uint4 w[N];
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const int k = v + T * u;
      w[u] = make_uint4(0u, 0u, 0u, 0u);
      if ((FULL || k < r.vecs) && ZS_CHECK(aligned(body + 16 * k, 16) && r.head + 8 * k + 8 <= len, 71, k))
        w[u] = ld16_behind(body + 16 * k);
    }
#pragma unroll
    for (int u = 0; u < N; ++u) g.template vec16<DT>(w[u]);
  }
}

// The partial of elements [0, len) at p, in thread 0.
template <int P, int DT, int T>
__device__ __forceinline__ double piece_sum(const void* p, int len, float2* red) {
  constexpr int es = SrcTraits<DT>::esize;
  constexpr int kAhead = (DT == ZERO_F32) ? kAhead32 : kAhead16;  // vectors in flight per thread
  const Run r = vector_run<es>(p, len);
  const char* body = static_cast<const char*>(p) + es * r.head;
  Gather<P> g;
  int v = thread_of<T>();
  for (; v + T * (kAhead - 1) < r.vecs; v += T * kAhead) gather_vectors<P, DT, T, kAhead, true>(body, v, r, len, g);
  for (; v < r.vecs; v += T * 4) gather_vectors<P, DT, T, 4, false>(body, v, r, len, g);
  const int e = ragged_element(r, len, thread_of<T>());
  if (e >= 0 && ZS_CHECK(e < len, 72, e)) g.template one<DT>(p, e);
  __syncwarp();
  if (P == ZERO_NORM_INF)
    return static_cast<double>(__uint_as_float(max_of<T>(g.template top<DT>(), reinterpret_cast<uint32_t*>(red))));
  const double sum = sum_norm<T>(g.acc, red);
  // Squares below 2^-126 have lost bits: at most 2^-150 each, 2^-133 of a
  // piece, so a sum of 2^-96 and more has lost at most 2^-37.  Magnitudes lose none.
  const bool fits = sum < static_cast<double>(INFINITY) && (P == ZERO_NORM_1 || sum >= 0x1p-96);
  if (!any_of<T>(thread_of<T>() == 0 && !fits)) return sum;
  if (P == ZERO_NORM_2 && !any_of<T>(g.template any<DT>())) return 0.0;
  return scaled_sum<P, DT, T>(p, len, red);
}

template <int P, int T>
__device__ __forceinline__ void piece_partial(const zero_grad_entry& t, const GradPiece& c, double* partials, float2* red) {
  if (!ZS_CHECK(c.len > 0 && c.k >= 0 && c.k + c.len <= t.numel, 73, c.at)) return;
  const char* src = static_cast<const char*>(t.src);
  double sum = 0.0;
  if (src != nullptr) {
    if (t.src_dtype == ZERO_F32)
      sum = piece_sum<P, ZERO_F32, T>(src + 4 * c.k, c.len, red);
    else if (t.src_dtype == ZERO_BF16)
      sum = piece_sum<P, ZERO_BF16, T>(src + 2 * c.k, c.len, red);
    else
      sum = piece_sum<P, ZERO_F16, T>(src + 2 * c.k, c.len, red);
  }
  if (thread_of<T>() == 0) partials[c.at] = sum;
}

template <int P>
__global__ void __launch_bounds__(kSumThreads, kSumBlocks)
    chunk_sums_kernel(const zero_grad_entry* __restrict__ entries, int n, const __grid_constant__ GradPlan plan,
                      double* __restrict__ partials) {
  __shared__ float2 red[kSumThreads / 32];
  const int block = blockIdx.x;
  let_next_start();
  if (block < plan.n_wide) {
    const GradPiece c = wide_piece(entries, n, plan, block);  // of the plan, not of what runs before
    wait_before();
    piece_partial<P, kSumThreads>(entries[c.tensor], c, partials, red);
  } else {
    const GradPiece c = narrow_piece<kSumThreads>(entries, plan, block);
    wait_before();
    if (c.len > 0) piece_partial<P, 32>(entries[c.tensor], c, partials, red);
  }
}

// ------------------------------------------ 2: tensors, groups and all
// The two ways of joining: sums, and the largest with NaN above all.
template <int P>
__device__ __forceinline__ double join(double a, double b) {
  if (P != ZERO_NORM_INF) return a + b;
  return (a > b || a != a) ? a : b;
}

// Lane 0's result, of the first `lanes` lanes.
template <int P>
__device__ __forceinline__ double warp_join(double x, int lanes = 32) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
    if (off < lanes) x = join<P>(x, __shfl_down_sync(0xffffffffu, x, off));
  return x;
}

constexpr int kFinishThreads = 1024;
constexpr int kFinishBlocks = 8;  // at most: one cluster

// Shared memory of a block that joins.
template <int T>
struct Joining {
  double buf[T];
  int queue[T];
  int queued;
};

// Thread 0's result; every thread of the block must call it.  A warp's
// binary64 addition takes 16 cycles whether for one lane or 32, so an eighth of
// the threads first adds eight values each.
template <int P, int T>
__device__ __forceinline__ double block_join(double x, double* buf) {
  constexpr int kAdding = T / 8;
  buf[threadIdx.x] = x;
  __syncthreads();
  if (threadIdx.x < kAdding) {
#pragma unroll
    for (int k = 1; k < 8; ++k) x = join<P>(x, buf[threadIdx.x + k * kAdding]);
    x = warp_join<P>(x);
  }
  __syncthreads();
  if (threadIdx.x < kAdding && (threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
  __syncthreads();
  if (threadIdx.x == 0)
#pragma unroll
    for (int w = 1; w < kAdding / 32; ++w) x = join<P>(x, buf[w]);
  __syncthreads();
  return x;
}

// The same where only the first few lanes of each warp have something (zeros
// in the others): fewer barriers.
template <int P, int T>
__device__ __forceinline__ double block_join_few(double x, int lanes, double* buf) {
  static_assert(T == 1024, "one value of a lane for each warp");
  x = warp_join<P>(x, lanes);
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
  __syncthreads();
  if (threadIdx.x < 32) x = warp_join<P>(buf[threadIdx.x]);
  __syncthreads();
  return x;
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
    for (int u = 0; u < 8; ++u)
      if (i + u * step < count) acc = join<P>(acc, v[u]);
  }
  return acc;
}

// A run of values up to which a thread joins it, and a warp; above, a block.
constexpr int kThreadRun = 16, kWarpRun = 1024;

// load(lo), ..., load(lo + count - 1) joined, each thread's own run; every
// thread of the block must call it.
template <int P, int T, class Load>
__device__ __forceinline__ double run_join(int lo, int count, const Load& load, Joining<T>& sh) {
  double s = 0.0;
  if (threadIdx.x == 0) sh.queued = 0;
  if (count <= kThreadRun) s = strided<P>(0, count, 1, [&](int j) { return load(lo + j); });
  unsigned mid = __ballot_sync(0xffffffffu, count > kThreadRun && count <= kWarpRun);
  for (; mid != 0u; mid &= mid - 1u) {
    const int l = __ffs(mid) - 1, from = __shfl_sync(0xffffffffu, lo, l), len = __shfl_sync(0xffffffffu, count, l);
    double x = warp_join<P>(strided<P>(threadIdx.x & 31, len, 32, [&](int j) { return load(from + j); }));
    x = __shfl_sync(0xffffffffu, x, 0);
    if ((threadIdx.x & 31) == l) s = x;
  }
  if (!__syncthreads_or(count > kWarpRun)) return s;
  int slot = 0;
  if (count > kWarpRun) sh.queue[slot = atomicAdd(&sh.queued, 1)] = threadIdx.x;  // their order does not matter
  __syncthreads();
  const int n = sh.queued;
  for (int q = 0; q < n; ++q) {
    // the run of the queued thread, by way of the buffer that block_join uses
    if (static_cast<int>(threadIdx.x) == sh.queue[q]) {
      reinterpret_cast<int*>(sh.buf)[0] = lo;
      reinterpret_cast<int*>(sh.buf)[1] = count;
    }
    __syncthreads();
    const int from = reinterpret_cast<int*>(sh.buf)[0], len = reinterpret_cast<int*>(sh.buf)[1];
    __syncthreads();
    const double x = block_join<P, T>(strided<P>(threadIdx.x, len, T, [&](int j) { return load(from + j); }), sh.buf);
    if (threadIdx.x == 0) sh.buf[0] = x;
    __syncthreads();
    if (count > kWarpRun && slot == q) s = sh.buf[0];
    __syncthreads();
  }
  return s;
}

struct FinishArgs {
  GradPlan plan;
  int n, n_groups;
  const double* partials;  // of the chunks; or the ranks' sums, n_parts rows of n
  int n_parts;
  float scale;
  const float* dscale;
  double* sums;            // of the tensors, over all parts
  const double* max_norms;
  float* norms;
  zero_norm_result* results;  // NULL: the sums only
  int32_t* found;
};

// Tensors, and groups, that finish_kernel takes.
constexpr int kFinishMost = 1024;
static_assert(kFinishMost <= kFinishThreads, "a thread of finish_kernel has at most one tensor and one group");
// Up to these one block finishes.
constexpr int kBlockTensors = 128, kBlockPartials = 2048, kBlockParts = 256;
// Partials up to which 8 lanes of tensors_kernel add a tensor's; above, a block.
constexpr int kOctetPartials = 512;

__device__ __forceinline__ void partials_of(const GradPlan& p, int i, int& lo, int& count) {
  const int j = __ldg(p.narrow_of + i);
  lo = j >= 0 ? p.n_wide + j : __ldg(p.first + i);
  count = j >= 0 ? 1 : __ldg(p.first + i + 1) - lo;
}

template <int P>
__device__ __forceinline__ double scale_power(const FinishArgs& a) {
  const double s = fabs(static_cast<double>(a.dscale != nullptr ? *a.dscale : a.scale));
  return P == ZERO_NORM_2 ? s * s : s;
}

template <int P>
__device__ __forceinline__ double join_parts(const FinishArgs& a, int i) {
  const double* const row = a.partials + i;
  return strided<P>(0, a.n_parts, 1, [&](int r) { return ld_behind(row + static_cast<int64_t>(r) * a.n); });
}

// Roots and quotients: binary32 ones corrected by Newton's method with binary64
// residuals, where the chain of binary64 operations of __dsqrt_rn and __ddiv_rn
// is much of the time that one thread takes for a result (a small list's norms 8.4
// against 7.8 us).  The root of s: y + (s - y y) / 2y twice.  With u = 2^-24, y is
// 1.5 u off at first (s and the root rounded) and the factor 1 / 2y u more, which leaves
// 1.125 u^2 + 1.5 u^2 after the first step and, after the second, what the last
// addition rounds.
__device__ __forceinline__ bool in_float_range(float f) { return f > 0x1p-100f && f < 0x1p100f; }
__device__ __forceinline__ double root(double s) {
  const float f = __double2float_rn(s);
  if (!in_float_range(f)) return __dsqrt_rn(s);
  const float y0 = __fsqrt_rn(f);
  const double half = static_cast<double>(__fdiv_rn(0.5f, y0));
  double y = static_cast<double>(y0);
  y = fma(fma(-y, y, s), half, y);
  return fma(fma(-y, y, s), half, y);
}
// A tensor's norm in binary32, at most u (1 + 2^-21) off: one such step, its residual and
// quotient rounded by u each, leaves 1.125 u^2 + 2 u x 1.5 u before the last rounding.
template <int P>
__device__ __forceinline__ float tensor_norm(double s) {
  const float f = __double2float_rn(s);
  if (P != ZERO_NORM_2) return f;
  if (!in_float_range(f)) return __double2float_rn(__dsqrt_rn(s));
  const float y = __fsqrt_rn(f);
  const float rest = __double2float_rn(fma(-static_cast<double>(y), static_cast<double>(y), s));
  return __fadd_rn(y, __fdiv_rn(rest, 2.0f * y));
}
// min(1, limit / d) in binary32, at most u (1 + 2^-20) off where it is above 2^-100: the
// first quotient is 3 u off (limit, d and itself rounded); residual, d and the second
// quotient, rounded by u each, leave 3 u x 3 u before the last rounding.
__device__ __forceinline__ float clip_coefficient(double limit, double d) {
  if (!(limit < d)) return 1.0f;  // a NaN too
  const float fd = __double2float_rn(d), fl = __double2float_rn(limit);
  if (!in_float_range(fd) || !in_float_range(fl)) return __double2float_rn(__ddiv_rn(limit, d));
  const float q = __fdiv_rn(fl, fd);
  const float rest = __double2float_rn(fma(-static_cast<double>(q), d, limit));
  return fminf(1.0f, __fadd_rn(q, __fdiv_rn(rest, fd)));
}

template <int P>
__device__ __forceinline__ void write_result(const FinishArgs& a, int g, double sum, double limit) {
  const double norm = P == ZERO_NORM_2 ? root(sum) : sum;
  zero_norm_result r;
  r.sqnorm = sum;
  r.norm = norm;
  r.clip_coef = g < a.n_groups ? clip_coefficient(limit, __dadd_rn(norm, 1e-6)) : 1.0f;
  r.finite = isfinite(norm) ? 1 : 0;
  if (g == a.n_groups && a.found != nullptr && !r.finite) *a.found = 1;
  a.results[g] = r;
  a.norms[a.n + g] = __double2float_rn(norm);
}
template <int P>
__device__ __forceinline__ void write_group(const FinishArgs& a, int g, double sum) {
  write_result<P>(a, g, sum, ld_behind(a.max_norms + g));
}

// The sums and norms of many tensors over all SMs (the binary64 pipes of
// finish_kernel's 8 SMs alone took 38 us for 20,000 tensors): 8 lanes for
// each, or a thread to join the ranks' sums.
template <int P, bool PARTS>
__global__ void __launch_bounds__(256) tensors_kernel(const __grid_constant__ FinishArgs a) {
  __shared__ double buf[256];
  let_next_start();
  if (PARTS) {
    wait_before();
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i >= a.n) return;
    const double s = join_parts<P>(a, i);
    a.sums[i] = s;
    a.norms[i] = tensor_norm<P>(s);
    return;
  }
  const int base = blockIdx.x * 32, i = base + (threadIdx.x >> 3), lane = threadIdx.x & 7;
  int lo = 0, count = 0;
  if (i < a.n) partials_of(a.plan, i, lo, count);  // of the plan: while the kernel before still runs
  wait_before();
  const double factor = scale_power<P>(a);
  const auto finish = [&](int k, double s) {
    s *= factor;
    a.sums[k] = s;
    if (a.norms != nullptr) a.norms[k] = tensor_norm<P>(s);
  };
  double s = 0.0;
  if (count <= kOctetPartials) s = strided<P>(lane, count, 8, [&](int j) { return ld_behind(a.partials + lo + j); });
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) s = join<P>(s, __shfl_down_sync(0xffffffffu, s, off, 8));
  if (lane == 0 && i < a.n && count <= kOctetPartials) finish(i, s);
  if (!__syncthreads_or(count > kOctetPartials)) return;
  for (int k = base; k < base + 32 && k < a.n; ++k) {
    partials_of(a.plan, k, lo, count);
    if (count <= kOctetPartials) continue;
    s = block_join<P, 256>(strided<P>(threadIdx.x, count, 256, [&](int j) { return ld_behind(a.partials + lo + j); }), buf);
    if (threadIdx.x == 0) finish(k, s);
  }
}

// The sum over all, from the blocks of a cluster, and its result (and that of
// a single group, which is the same); `all`: this thread's part of it, where
// lanes > 0 in that many lanes of a warp.  The barriers also order what the
// blocks have written.
template <int P>
__device__ __forceinline__ void finish_all(const FinishArgs& a, double all, int lanes, Joining<kFinishThreads>& sh,
                                           double* total, int blocks) {
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank()), lane = threadIdx.x & 31;
  all = lanes > 0 ? block_join_few<P, kFinishThreads>(all, lanes, sh.buf) : block_join<P, kFinishThreads>(all, sh.buf);
  if (blocks > 1) {
    if (threadIdx.x == 0) *total = all;
    cluster.sync();
    if (rank == 0 && threadIdx.x < 32) {
      all = lane < blocks ? *cluster.map_shared_rank(total, lane) : 0.0;
      all = warp_join<P>(all, blocks);
    }
  }
  if (rank == 0 && threadIdx.x == 0) {
    write_result<P>(a, a.n_groups, all, 0.0);
    if (a.n_groups == 1) write_group<P>(a, 0, all);
  }
}

// Group g of a thread (-1: none): its tensors' sums joined, its result.
template <int P>
__device__ __forceinline__ void finish_group(const FinishArgs& a, int g, int lo, int count, Joining<kFinishThreads>& sh) {
  const double s = run_join<P, kFinishThreads>(
      lo, count, [&](int j) { return ld_behind(a.sums + __ldg(a.plan.members + j)); }, sh);
  if (g >= 0) write_group<P>(a, g, s);
}
__device__ __forceinline__ void members_of(const GradPlan& p, int g, int& lo, int& count) {
  lo = count = 0;
  if (g < 0) return;
  lo = __ldg(p.group_first + g);
  count = __ldg(p.group_first + g + 1) - lo;
}

// Whether most groups' sums are a thread's work: then as few warps as hold the
// groups make them, since a result's binary64 operations take a warp as long
// for one group as for 32; else the groups spread over the warps.
__device__ __forceinline__ bool few_members(const FinishArgs& a) { return a.n / a.n_groups < kThreadRun; }

// Up to 1024 tensors and groups: one cluster of 8 blocks, or one block.  Of its
// W warps tensor i belongs to warp i % W, lane i / W: long tensors, whose
// partials a warp or a block adds, spread over the warps.  (PARTS: as few
// warps as hold the tensors.)
template <int P, bool PARTS>
__global__ void __launch_bounds__(kFinishThreads) finish_kernel(const __grid_constant__ FinishArgs a) {
  __shared__ Joining<kFinishThreads> sh;
  __shared__ double total;
  const int blocks = gridDim.x, warps = blocks * (kFinishThreads / 32), rank = blockIdx.x;
  const int spread = (threadIdx.x & 31) * warps + (threadIdx.x >> 5) * blocks + rank, dense = threadIdx.x * blocks + rank;
  const int i = PARTS ? dense : spread, k = few_members(a) ? dense : spread;
  const int g = a.n_groups > 1 && k < a.n_groups ? k : -1;
  let_next_start();
  // of the plan: while the kernel before still runs
  int lo = 0, count = 0, group_lo, group_count;
  if (!PARTS && i < a.n) partials_of(a.plan, i, lo, count);
  members_of(a.plan, g, group_lo, group_count);
  wait_before();
  double s = 0.0;
  if (PARTS) {
    if (i < a.n) s = join_parts<P>(a, i);
  } else {
    s = run_join<P, kFinishThreads>(lo, count, [&](int j) { return ld_behind(a.partials + j); }, sh) * scale_power<P>(a);
  }
  if (i < a.n) {
    a.sums[i] = s;
    if (a.norms != nullptr) a.norms[i] = tensor_norm<P>(s);
  }
  if (a.results == nullptr) return;
  finish_all<P>(a, i < a.n ? s : 0.0, PARTS ? 0 : (a.n + warps - 1) / warps, sh, &total, blocks);
  if (a.n_groups > 1) finish_group<P>(a, g, group_lo, group_count, sh);
  if (blocks > 1) cg::this_cluster().sync();  // total is read until here
}

// More of either: the first cluster makes the result over all, the other
// blocks those of `per` groups each.
template <int P>
__global__ void __launch_bounds__(kFinishThreads) groups_kernel(const __grid_constant__ FinishArgs a, int per) {
  __shared__ Joining<kFinishThreads> sh;
  __shared__ double total;
  let_next_start();
  if (blockIdx.x < kFinishBlocks) {
    wait_before();
    const int at = blockIdx.x * kFinishThreads + threadIdx.x;
    const double s = strided<P>(at, a.n, kFinishBlocks * kFinishThreads, [&](int j) { return ld_behind(a.sums + j); });
    finish_all<P>(a, s, 0, sh, &total, kFinishBlocks);
    cg::this_cluster().sync();  // total is read until here
  } else {
    const int k = few_members(a) ? threadIdx.x : (threadIdx.x & 31) * (kFinishThreads / 32) + (threadIdx.x >> 5);
    const int64_t at = static_cast<int64_t>(blockIdx.x - kFinishBlocks) * per + k;
    const int g = k < per && at < a.n_groups ? static_cast<int>(at) : -1;
    int lo, count;
    members_of(a.plan, g, lo, count);
    wait_before();
    finish_group<P>(a, g, lo, count, sh);
  }
}

// -------------------------------------------------------------- launches
template <int P, bool PARTS>
static zero_status launch_finish(const FinishArgs& k, cudaStream_t st) {
  const bool small = k.n <= kFinishMost, whole = small && (k.n_groups <= kFinishMost || k.results == nullptr);
  zero_status s = ZERO_OK;
  if (small) {
    const bool few = PARTS ? k.n <= kBlockParts : k.n <= kBlockTensors && k.plan.n_wide + k.plan.n_narrow <= kBlockPartials;
    const unsigned blocks = few ? 1 : kFinishBlocks;
    FinishArgs f = k;
    if (!whole) f.results = nullptr;
    s = launch_after("finish_kernel", finish_kernel<P, PARTS>, blocks, kFinishThreads, blocks, st, f);
  } else {
    s = launch_after("tensors_kernel", tensors_kernel<P, PARTS>, one_pass_blocks(k.n, PARTS ? 256 : 32), 256, 1, st, k);
  }
  if (s != ZERO_OK || whole || k.results == nullptr) return s;
  int per = 0;
  unsigned blocks = kFinishBlocks;
  if (k.n_groups > 1) {  // over the SMs, in whole clusters
    per = k.n_groups <= 144 ? 1 : k.n_groups >= 144 * kFinishThreads ? kFinishThreads : (k.n_groups + 143) / 144;
    const unsigned need = one_pass_blocks(k.n_groups, per);
    blocks += (need + kFinishBlocks - 1) / kFinishBlocks * kFinishBlocks;
  }
  return launch_after("groups_kernel", groups_kernel<P>, blocks, kFinishThreads, kFinishBlocks, st, k, per);
}

template <int P>
static zero_status launch_norms_t(const GradListArgs& a, double* partials, const FinishArgs& k, cudaStream_t st) {
  if (grad_blocks(k.plan, kSumThreads) > 0) {
    const zero_status s = launch_after("chunk_sums_kernel", chunk_sums_kernel<P>, grad_blocks(k.plan, kSumThreads),
                                       kSumThreads, 1, st, a.entries, a.n, k.plan, partials);
    if (s != ZERO_OK) return s;
  }
  return launch_finish<P, false>(k, st);
}

ZS_DEBUG_UNIT(list_norms)

zero_status launch_list_norms(const GradListArgs& a, double* partials, double* sums, const double* max_norms, float* norms,
                              zero_norm_result* results, int32_t* found, cudaStream_t st) {
  const FinishArgs k{plan_parts(a), a.n, a.n_groups, partials, 1, a.scale, a.dscale, sums,
                     max_norms, norms, results, found};
  if (a.norm_type == ZERO_NORM_2) return launch_norms_t<ZERO_NORM_2>(a, partials, k, st);
  if (a.norm_type == ZERO_NORM_1) return launch_norms_t<ZERO_NORM_1>(a, partials, k, st);
  return launch_norms_t<ZERO_NORM_INF>(a, partials, k, st);
}

zero_status launch_sums_norms(const GradListArgs& a, const double* sums, int n_parts, double* joined,
                              const double* max_norms, float* norms, zero_norm_result* results, int32_t* found,
                              cudaStream_t st) {
  const FinishArgs k{plan_parts(a), a.n, a.n_groups, sums, n_parts, 1.0f, nullptr, joined,
                     max_norms, norms, results, found};
  if (a.norm_type == ZERO_NORM_2) return launch_finish<ZERO_NORM_2, true>(k, st);
  if (a.norm_type == ZERO_NORM_1) return launch_finish<ZERO_NORM_1, true>(k, st);
  return launch_finish<ZERO_NORM_INF, true>(k, st);
}

}  // namespace zs
