// list_clip.cu -- the grads of a list, scaled and clipped by their groups'
// coefficients, in place or into buffers of another type.
//
// y = fl_type(fl(f x)), f = fl(scale * coef): a rounding to binary32 and, for
// 16-bit outputs, one to their type (both to nearest even).
//
// Up to 8 blocks per wide chunk, one warp per narrow tensor (list_norms.cu's
// work split), the last first: the norms pass has just read the list front to
// back, and its end may be in L2 (128 MB in place 37.9 us, front to back 39.9).
// Nothing is written where the norm over all tensors is not finite, nor in
// place where scale and coefficient are 1.
//
// Bound by HBM: 1.88e9 bf16 elements in place 1056 us = 7.1 TB/s, 302e6 fp16
// into fp32 264 us = 6.9 TB/s; 2^28 fp16 into fp32 whose place on the vector
// grid is another one, element by element, 877 to 913 us = 1.8 TB/s.  What lies in L2 is no faster: 32 to 64 MB read and
// written there at 7.5 to 8 TB/s.
#include "common.cuh"
#include "grad_list.cuh"
#include "kernels.h"

namespace zs {

constexpr int kClipThreads = 256, kClipBlocks = 4;
// Elements of a wide chunk that a block clips: fewer than the chunk has, so that
// the blocks in flight read and write fewer places of memory at once (eight
// layers of Llama-7B in bf16, 7.5 GB: 1056 us with 16384, 1067 with 32768, 1084
// with 65536, 1139 with 8192).
constexpr int kClipPiece = 16384;

// 16 bytes that this thread overwrites later.
__device__ __forceinline__ uint4 ld16_rw(const void* p) {
  uint4 r;
  asm volatile("ld.global.cs.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
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

// N vectors of 8, T apart, from number v on, all loaded before the first is
// stored; those from r.vecs on are left out unless FULL.
template <int S, int D, int T, int N, bool FULL>
__device__ __forceinline__ void clip_vectors(const char* from, char* to, int v, const Run& r, int len, float f) {
  constexpr int se = SrcTraits<S>::esize, de = SrcTraits<D>::esize;
  Vec8<S> x[N];
#pragma unroll
  for (int u = 0; u < N; ++u) {
    const int k = v + T * u;
    if ((FULL || k < r.vecs) && ZS_CHECK(aligned(from + 8 * se * k, 8 * se) && r.head + 8 * k + 8 <= len, 75, k))
      x[u].load(from + 8 * se * k);
  }
#pragma unroll
  for (int u = 0; u < N; ++u) {
    const int k = v + T * u;
    if ((FULL || k < r.vecs) && ZS_CHECK(aligned(to + 8 * de * k, 8 * de) && r.head + 8 * k + 8 <= len, 76, k)) {
      float y[8];
      x[u].widen(y);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = __fmul_rn(f, y[j]);
      store8<D>(to + 8 * de * k, y);
    }
  }
}

template <int S, int D, int T>
__device__ __forceinline__ void clip_piece(const char* src, char* dst, int len, float f, int thread) {
  constexpr int se = SrcTraits<S>::esize, de = SrcTraits<D>::esize;
  constexpr int kAhead = (S == ZERO_F32) ? 4 : 8;
  const Run r = vector_run<se>(src, len);
  const char* from = src + se * r.head;
  char* to = dst + de * r.head;
  if (aligned(to, 8 * de)) {
    int v = thread;
    for (; v + T * (kAhead - 1) < r.vecs; v += T * kAhead) clip_vectors<S, D, T, kAhead, true>(from, to, v, r, len, f);
    for (; v < r.vecs; v += T * 4) clip_vectors<S, D, T, 4, false>(from, to, v, r, len, f);
    const int e = ragged_element(r, len, thread);
    if (e >= 0 && ZS_CHECK(e < len, 77, e)) store_one<D>(dst, e, __fmul_rn(f, elem_behind<S>(src, e)));
  } else {  // source and destination apart on the vector grid: element by element
#pragma unroll 8
    for (int e = thread; e < len; e += T) store_one<D>(dst, e, __fmul_rn(f, elem_behind<S>(src, e)));
  }
}

template <int D, int T>
__device__ __forceinline__ void clip_to(int src_dtype, const char* src, char* dst, int len, float f, int thread) {
  if (src == nullptr) {
    for (int e = thread; e < len; e += T) store_one<D>(dst, e, 0.0f);
  } else if (src_dtype == ZERO_F32) {
    clip_piece<ZERO_F32, D, T>(src, dst, len, f, thread);
  } else if (src_dtype == ZERO_BF16) {
    clip_piece<ZERO_BF16, D, T>(src, dst, len, f, thread);
  } else {
    clip_piece<ZERO_F16, D, T>(src, dst, len, f, thread);
  }
}

template <int T>
__device__ __forceinline__ void clip_tensor(const zero_grad_entry& t, const GradPiece& c, int n_groups, float scale,
                                            const zero_norm_result* results) {
  if (t.dst == nullptr) return;
  if (!ZS_CHECK(c.len > 0 && c.k >= 0 && c.k + c.len <= t.numel && t.group >= 0 && t.group < n_groups, 78, c.at)) return;
  const float coef = results[t.group].clip_coef;
  if (t.dst == t.src && coef == 1.0f && scale == 1.0f) return;
  const float f = __fmul_rn(scale, coef);
  const int thread = T == 32 ? threadIdx.x & 31 : threadIdx.x;
  const char* src = t.src == nullptr ? nullptr : static_cast<const char*>(t.src) + (t.src_dtype == ZERO_F32 ? 4 : 2) * c.k;
  char* dst = static_cast<char*>(t.dst) + (t.dst_dtype == ZERO_F32 ? 4 : 2) * c.k;
  if (t.dst_dtype == ZERO_F32)
    clip_to<ZERO_F32, T>(t.src_dtype, src, dst, c.len, f, thread);
  else if (t.dst_dtype == ZERO_BF16)
    clip_to<ZERO_BF16, T>(t.src_dtype, src, dst, c.len, f, thread);
  else
    clip_to<ZERO_F16, T>(t.src_dtype, src, dst, c.len, f, thread);
}

// The grid, from its end: the blocks of the narrow tensors, then 2^share blocks
// for each wide chunk.  MAY_LEAVE (in place with a scale of 1): the blocks look
// first whether any group is to be clipped; a chunk has one block then, as
// leaving takes 0.7 ns a block.  Where they stay, 1.88e9 bf16 elements take 36
// to 40 us more than in blocks of kClipPiece (norms and clip 1633 to 1641 against 1597
// to 1601), 377e6 fp32 5 to 6 (670 against 664), GPT-2's 124e6 bf16 up to 1 (138 against 137).
template <bool MAY_LEAVE>
__global__ void __launch_bounds__(kClipThreads, kClipBlocks)
    list_clip_kernel(const zero_grad_entry* __restrict__ entries, int n, int n_groups,
                     const __grid_constant__ GradPlan plan, int share, float scale, const float* dscale,
                     const zero_norm_result* results) {
  const int block = gridDim.x - 1 - blockIdx.x, wide_blocks = plan.n_wide << share;
  GradPiece c;
  if (!MAY_LEAVE && block < wide_blocks) c = wide_piece(entries, n, plan, block >> share);  // while the kernel before still runs
  wait_before();
  if (!results[n_groups].finite) return;
  if (MAY_LEAVE && n_groups <= 32) {
    const int g = threadIdx.x & 31;
    if (__all_sync(0xffffffffu, g >= n_groups || results[g].clip_coef == 1.0f)) return;
  }
  if (dscale != nullptr) scale = *dscale;
  if (block < wide_blocks) {
    if (MAY_LEAVE) c = wide_piece(entries, n, plan, block >> share);
    const int piece = plan.chunk >> share, skip = (block & ((1 << share) - 1)) * piece;
    c.k += skip;
    c.len = min(c.len - skip, piece);
    if (c.len > 0) clip_tensor<kClipThreads>(entries[c.tensor], c, n_groups, scale, results);
  } else {
    c = narrow_piece<kClipThreads>(entries, plan, block - wide_blocks + plan.n_wide);
    if (c.len > 0) clip_tensor<32>(entries[c.tensor], c, n_groups, scale, results);
  }
}

ZS_DEBUG_UNIT(list_clip)

zero_status launch_list_clip(const GradListArgs& a, const zero_norm_result* results, cudaStream_t st) {
  const GradPlan plan = plan_parts(a);
  const int64_t narrow = grad_blocks(plan, kClipThreads) - static_cast<unsigned>(plan.n_wide);
  const bool may_leave = a.in_place && a.dscale == nullptr && a.scale == 1.0f;
  int share = 0;
  if (!may_leave)
    while ((plan.chunk >> share) > kClipPiece) ++share;
  const int64_t blocks = (static_cast<int64_t>(plan.n_wide) << share) + narrow;
  if (blocks > 0x7fffffffLL) return fail(ZERO_EINVAL, "zero_list_clip: %lld blocks", (long long)blocks);
  if (blocks == 0) return ZERO_OK;
  return launch_after("list_clip_kernel", may_leave ? list_clip_kernel<true> : list_clip_kernel<false>,
                      static_cast<unsigned>(blocks), kClipThreads, 1, st, a.entries, a.n, a.n_groups, plan, share,
                      a.scale, a.dscale, results);
}

}  // namespace zs
