// list_clip.cu -- the grads of a list, scaled and clipped by their groups'
// coefficients, in place or into buffers of another type.
//
// y = fl_type(fl(f x)), f = fl(scale * coef): a rounding to binary32 and, for
// 16-bit outputs, one to their type (both to nearest even).
//
// One block per chunk (list_norms.cu's chunks), the last chunk first: the
// norms pass has just read the list front to back, so its end is what the
// 129 MB L2 still holds.  Nothing is written where the norm over all tensors
// is not finite, nor in place where scale and coefficient are 1.
#include "common.cuh"
#include "grad_list.cuh"
#include "kernels.h"

namespace zs {

// 16 bytes that this thread may overwrite later: a coherent load.
__device__ __forceinline__ uint4 ld16_rw(const void* p) {
  uint4 r;
  asm volatile("ld.global.cs.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}

template <int DT>
__device__ __forceinline__ float load_rw(const void* p, int e) {
  if (DT == ZERO_F32) return static_cast<const volatile float*>(p)[e];
  return half_bits_to_f32<DT>(static_cast<const volatile unsigned short*>(p)[e]);
}

template <int DT>
__device__ __forceinline__ void store_one(void* p, int e, float y) {
  if (DT == ZERO_F32)
    static_cast<float*>(p)[e] = y;
  else
    static_cast<unsigned short*>(p)[e] = round1_rn<DT>(y);
}

// 8 elements as loaded
template <int DT>
struct Vec8 {
  uint4 w;
  __device__ __forceinline__ void load(const char* p) { w = ld16_rw(p); }
  __device__ __forceinline__ void widen(float (&x)[8]) const {
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = half_bits_to_f32<DT>(ws[j] & 0xffffu);
      x[2 * j + 1] = half_bits_to_f32<DT>(ws[j] >> 16);
    }
  }
};
template <>
struct Vec8<ZERO_F32> {
  float v[8];
  __device__ __forceinline__ void load(const char* p) { ld8_rw(reinterpret_cast<const float*>(p), v); }
  __device__ __forceinline__ void widen(float (&x)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = v[j];
  }
};

template <int DT>
__device__ __forceinline__ void store8(char* p, const float (&y)[8]) {
  if constexpr (DT == ZERO_F32)
    st8(reinterpret_cast<float*>(p), y);
  else
    st16(p, make_uint4(pack2_rn<DT>(y[0], y[1]), pack2_rn<DT>(y[2], y[3]), pack2_rn<DT>(y[4], y[5]),
                       pack2_rn<DT>(y[6], y[7])));
}

template <int S, int D>
__device__ __forceinline__ void clip_chunk(const char* src, char* dst, int len, float f) {
  constexpr int se = SrcTraits<S>::esize, de = SrcTraits<D>::esize;
  constexpr int kAhead = (S == ZERO_F32) ? 4 : 8;
  const Run r = vector_run<se>(src, len);
  if (aligned(dst + de * r.head, 8 * de)) {
    const char* from = src + se * r.head;
    char* to = dst + de * r.head;
    for (int v0 = threadIdx.x; v0 < r.vecs; v0 += kAhead * kGradThreads) {
      Vec8<S> x[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int v = v0 + u * kGradThreads;
        if (v < r.vecs && ZS_CHECK(aligned(from + 8 * se * v, 8 * se) && r.head + 8 * v + 8 <= len, 75, v))
          x[u].load(from + 8 * se * v);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int v = v0 + u * kGradThreads;
        if (v < r.vecs && ZS_CHECK(aligned(to + 8 * de * v, 8 * de) && r.head + 8 * v + 8 <= len, 76, v)) {
          float y[8];
          x[u].widen(y);
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = __fmul_rn(f, y[j]);
          store8<D>(to + 8 * de * v, y);
        }
      }
    }
    const int e = ragged_element(r, len);
    if (e >= 0 && ZS_CHECK(e < len, 77, e)) store_one<D>(dst, e, __fmul_rn(f, load_rw<S>(src, e)));
  } else {  // source and destination apart on the vector grid: element by element
#pragma unroll 8
    for (int e = threadIdx.x; e < len; e += kGradThreads) store_one<D>(dst, e, __fmul_rn(f, load_rw<S>(src, e)));
  }
}

template <int D>
__device__ __forceinline__ void clip_to(int src_dtype, const char* src, char* dst, int len, float f) {
  if (src == nullptr) {
    for (int e = threadIdx.x; e < len; e += kGradThreads) store_one<D>(dst, e, 0.0f);
  } else if (src_dtype == ZERO_F32) {
    clip_chunk<ZERO_F32, D>(src, dst, len, f);
  } else if (src_dtype == ZERO_BF16) {
    clip_chunk<ZERO_BF16, D>(src, dst, len, f);
  } else {
    clip_chunk<ZERO_F16, D>(src, dst, len, f);
  }
}

__global__ void __launch_bounds__(kGradThreads)
    list_clip_kernel(const zero_grad_entry* __restrict__ entries, int n, int n_groups,
                     const int32_t* __restrict__ first, int chunk, float scale, const float* __restrict__ dscale,
                     const zero_norm_result* __restrict__ results) {
  if (!results[n_groups].finite) return;
  if (dscale != nullptr) scale = *dscale;
  const GradChunk c = grad_chunk(entries, first, n, chunk, gridDim.x - 1 - blockIdx.x);
  const zero_grad_entry t = entries[c.tensor];
  if (t.dst == nullptr) return;
  if (!ZS_CHECK(c.len > 0 && c.k >= 0 && c.k + c.len <= t.numel && t.group >= 0 && t.group < n_groups, 78, blockIdx.x))
    return;
  const float coef = results[t.group].clip_coef;
  if (t.dst == t.src && coef == 1.0f && scale == 1.0f) return;
  const float f = __fmul_rn(scale, coef);
  const char* src = t.src == nullptr ? nullptr : static_cast<const char*>(t.src) + (t.src_dtype == ZERO_F32 ? 4 : 2) * c.k;
  char* dst = static_cast<char*>(t.dst) + (t.dst_dtype == ZERO_F32 ? 4 : 2) * c.k;
  if (t.dst_dtype == ZERO_F32)
    clip_to<ZERO_F32>(t.src_dtype, src, dst, c.len, f);
  else if (t.dst_dtype == ZERO_BF16)
    clip_to<ZERO_BF16>(t.src_dtype, src, dst, c.len, f);
  else
    clip_to<ZERO_F16>(t.src_dtype, src, dst, c.len, f);
}

ZS_DEBUG_UNIT(list_clip)

zero_status launch_list_clip(const GradListArgs& a, const zero_norm_result* results, cudaStream_t st) {
  if (a.n_chunks == 0) return ZERO_OK;
  list_clip_kernel<<<a.n_chunks, kGradThreads, 0, st>>>(a.entries, a.n, a.n_groups, a.plan, a.chunk, a.scale, a.dscale,
                                                        results);
  return check_launch("list_clip_kernel");
}

}  // namespace zs
