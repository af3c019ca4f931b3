// list.cuh -- what the two kernels over a list of separate tensors share:
// finding a chunk's tensor, the scalars of its group and a block's grads.
// Internal.
#pragma once

#include "state8.cuh"
#include "table.cuh"

namespace zs {

// The tensor of chunk c: the last i with first[i] <= c.  The warp's 32 lanes
// test 32 evenly spaced candidates a round (find_tensor_warp of table.cuh)
// until 128 are left, and those at once, four each: 1 round for up to 128
// tensors, 2 for 4096, 3 for 131072.  (32 candidates to the end, 75 tensors,
// 1.88e9 elements in 8 bits: 4.53 against 4.43 ms, 4000 tensors, 302e6: 0.804
// against 0.792; 128 candidates in every round: 0.810.)  first[] is 4 bytes
// a tensor and stays in the SM's L1; a map with one entry per chunk, a
// single read but from L2 or HBM, left blocks waiting longer before their
// first load (1.88e9 elements: 4.84 against 4.76 ms; 4000 ragged fp32 tensors:
// 1.29 against 1.27).
__device__ __forceinline__ int find_chunk_tensor(const int32_t* __restrict__ first, int n, int c) {
  const int lane = threadIdx.x & 31;
  int lo = 0, span = n;  // first[lo] <= c, the answer is in [lo, lo + span)
  while (span > 128) {
    const int step = (span + 31) >> 5;
    const int off = lane * step;
    const bool le = off < span && __ldg(first + lo + off) <= c;
    const int j = 31 - __clz(__ballot_sync(0xffffffffu, le));
    lo += j * step;
    span = min(step, span - j * step);
  }
  int le = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int off = 32 * q + lane;
    if (off < span && __ldg(first + lo + off) <= c) ++le;
  }
  return lo + __reduce_add_sync(0xffffffffu, le) - 1;
}

// Found by one warp for the block; every thread must call it.  (Each warp for
// itself: 30 instructions times four, 4566 against 4535 us for 1.88e9 elements
// in 8 bits.)
__device__ __forceinline__ int block_tensor(const int32_t* __restrict__ first, int n, int c) {
  __shared__ int found;
  if (threadIdx.x < 32) {
    const int ti = find_chunk_tensor(first, n, c);
    if (threadIdx.x == 0) found = ti;
  }
  __syncthreads();
  return found;
}

// The scalars of a tensor's group: the launch's, or those of the device step
// states; false: the prepared step is skipped.
__device__ __forceinline__ bool group_scalars(const ListScalars& hs, const zero_adamw_device_state* ds, int g,
                                              AdamScalars& s) {
  if (ds != nullptr) return step_scalars<true>(s, ds + g, s);
  s = hs.s[g];
  return true;
}

// This lane's 8 grads fl(scale * x) of the block that starts at element k of
// the tensor `src` (NULL: no grad, zeros); `left`: its elements from k on.  A
// 16-bit source off the 16-byte grid (a view of a flat grad) is realigned in
// registers where the vectors around the block lie inside the tensor, else
// read element by element, 8 consecutive ones per lane.
template <int DT, bool VEC>
__device__ __forceinline__ void load_block_grad(const void* src, int64_t k, int64_t left, float scale, float (&g)[8]) {
  constexpr int es = SrcTraits<DT>::esize;
  constexpr int vb = (DT == ZERO_F32) ? 32 : 16;
  const char* p = static_cast<const char*>(src) + es * k;
  if (src == nullptr) {
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = 0.0f;
  } else if (VEC && aligned(p, vb)) {
    load8_src<DT>(p + es * elem_of<VEC>(0), g);
  } else if (VEC && DT != ZERO_F32 && k >= 8 && left >= kBlock8 + 8) {
    float x[1][8];
    load8_shifted<DT, 1>(p - es * kBlock8 * (threadIdx.x >> 5), x);  // it counts from the thread block's first warp
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = x[0][j];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = (VEC || elem_of<VEC>(j) < left) ? load_elem<DT>(p, elem_of<VEC>(j)) : 0.0f;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) g[j] = __fmul_rn(scale, g[j]);
}

}  // namespace zs
