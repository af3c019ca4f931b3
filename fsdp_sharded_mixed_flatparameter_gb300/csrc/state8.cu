// state8.cu -- the fp32 moments of a flat shard (or of one tensor) into the
// 8-bit format of state8.cuh and back: a checkpoint in 32 bits, a run that
// goes on in 8.  A warp per block of 256 elements; 8 + 2 bytes per element
// either way, HBM-bound: pack 400e6 elements 0.549 ms = 7.30 TB/s (0.648 at
// four blocks per SM instead of six; seven spill: 0.741), unpack 1.63e9 2.32 ms
// = 7.03 TB/s; 15.6e6 elements 26 us either way.
#include "common.cuh"
#include "kernels.h"
#include "state8.cuh"

namespace zs {

template <bool VEC>
__device__ __forceinline__ void pack_block(const float* __restrict__ m, const float* __restrict__ v,
                                           const zero_state8& q, int64_t b, int left) {
  const int64_t k = b * kBlock8;
  if (!ZS_CHECK(left > 0 && (!VEC || (aligned(m + k, 32) && aligned(v + k, 32) && aligned(q.exp_avg + k, 8) &&
                                      aligned(q.root + k, 8))),
                80, k))
    return;
  float x[8], r[8];
  load_block_f32<VEC>(m + k, left, x);
  load_block_f32<VEC>(v + k, left, r);
  F2 xm[4], xr[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    xm[i] = pair(x[2 * i], x[2 * i + 1]);
    xr[i] = pair(__fsqrt_rn(r[2 * i]), __fsqrt_rn(r[2 * i + 1]));
  }
  uint2 cm, cr;
  float sm, sr;
  encode_block<VEC, kNearest>(xm, xr, warp_amax(xm), warp_amax(xr), 0u, 0, cm, cr, sm, sr, false, false,
                              false);
  store_codes<VEC>(q.exp_avg + k, left, cm);
  store_codes<VEC>(q.root + k, left, cr);
  if ((threadIdx.x & 31) == 0) {
    q.exp_avg_scale[b] = sm;
    q.root_scale[b] = sr;
  }
}

template <bool VEC>
__device__ __forceinline__ void unpack_block(const zero_state8& q, float* __restrict__ m, float* __restrict__ v,
                                             int64_t b, int left) {
  const int64_t k = b * kBlock8;
  if (!ZS_CHECK(left > 0 && (!VEC || (aligned(m + k, 32) && aligned(v + k, 32) && aligned(q.exp_avg + k, 8) &&
                                      aligned(q.root + k, 8))),
                81, k))
    return;
  const uint2 cm = load_codes<VEC>(q.exp_avg + k, left), cr = load_codes<VEC>(q.root + k, left);
  F2 xm[4], xr[4];
  float x[8], r[8];
  const float sm = q.exp_avg_scale[b], sr = q.root_scale[b];
  decode8(cm, xm);
  decode8(cr, xr);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const F2 y = mul2(xr[i], both(sr));
    unpair(mul2(xm[i], both(sm)), x[2 * i], x[2 * i + 1]);
    unpair(mul2(y, y), r[2 * i], r[2 * i + 1]);
  }
  store_block_f32<VEC>(m + k, left, x);
  store_block_f32<VEC>(v + k, left, r);
}

__global__ void __launch_bounds__(256, 6)
    state8_pack_kernel(const float* __restrict__ m, const float* __restrict__ v, int64_t n, zero_state8 q, bool vec) {
  const int64_t nb = (n + kBlock8 - 1) / kBlock8;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * 8;
  for (int64_t b = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); b < nb; b += stride) {
    const int64_t left = n - b * kBlock8;
    if (vec && left >= kBlock8)
      pack_block<true>(m, v, q, b, kBlock8);
    else
      pack_block<false>(m, v, q, b, static_cast<int>(left < kBlock8 ? left : kBlock8));
  }
}

__global__ void __launch_bounds__(256, 6)
    state8_unpack_kernel(zero_state8 q, int64_t n, float* __restrict__ m, float* __restrict__ v, bool vec) {
  const int64_t nb = (n + kBlock8 - 1) / kBlock8;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * 8;
  for (int64_t b = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); b < nb; b += stride) {
    const int64_t left = n - b * kBlock8;
    if (vec && left >= kBlock8)
      unpack_block<true>(q, m, v, b, kBlock8);
    else
      unpack_block<false>(q, m, v, b, static_cast<int>(left < kBlock8 ? left : kBlock8));
  }
}

static bool state8_vec(const float* m, const float* v, const zero_state8& q) {
  return aligned(m, 32) && aligned(v, 32) && aligned(q.exp_avg, 8) && aligned(q.root, 8);
}

ZS_DEBUG_UNIT(state8)

zero_status launch_state8_pack(const float* m, const float* v, int64_t n, const zero_state8& q, cudaStream_t st) {
  state8_pack_kernel<<<one_pass_blocks(n, 8 * kBlock8), 256, 0, st>>>(m, v, n, q, state8_vec(m, v, q));
  return check_launch("state8_pack_kernel");
}

zero_status launch_state8_unpack(const zero_state8& q, int64_t n, float* m, float* v, cudaStream_t st) {
  state8_unpack_kernel<<<one_pass_blocks(n, 8 * kBlock8), 256, 0, st>>>(q, n, m, v, state8_vec(m, v, q));
  return check_launch("state8_unpack_kernel");
}

}  // namespace zs
