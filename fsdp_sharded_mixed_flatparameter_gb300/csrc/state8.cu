// state8.cu -- the fp32 moments of a flat shard (or of one tensor) into the
// 8-bit format of state8.cuh and back: a checkpoint in 32 bits, a run that
// goes on in 8.  A warp per block of 256 elements; 8 + 2 bytes per element
// either way, HBM-bound.
#include "common.cuh"
#include "kernels.h"
#include "state8.cuh"

namespace zs {

__global__ void __launch_bounds__(256)
    state8_pack_kernel(const float* __restrict__ m, const float* __restrict__ v, int64_t n, zero_state8 q, bool vec) {
  const int64_t nb = (n + kBlock8 - 1) / kBlock8;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * 8;
  for (int64_t b = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); b < nb; b += stride) {
    const int64_t k = b * kBlock8;
    const int left = static_cast<int>(n - k < kBlock8 ? n - k : kBlock8);
    const bool w = vec && left == kBlock8;
    if (!ZS_CHECK(left > 0 && (!w || (aligned(m + k, 32) && aligned(v + k, 32) && aligned(q.exp_avg + k, 8) &&
                                      aligned(q.root + k, 8))),
                  80, k))
      continue;
    float x[8], r[8];
    load_block_f32(m + k, w, left, x);
    load_block_f32(v + k, w, left, r);
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = __fsqrt_rn(r[j]);
    uint32_t cm[2], cr[2];
    float sm, sr;
    encode_block<false>(x, r, w, 0u, 0, cm, cr, sm, sr);
    store_codes(q.exp_avg + k, w, left, cm);
    store_codes(q.root + k, w, left, cr);
    if ((threadIdx.x & 31) == 0) {
      q.exp_avg_scale[b] = sm;
      q.root_scale[b] = sr;
    }
  }
}

__global__ void __launch_bounds__(256)
    state8_unpack_kernel(zero_state8 q, int64_t n, float* __restrict__ m, float* __restrict__ v, bool vec) {
  const int64_t nb = (n + kBlock8 - 1) / kBlock8;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * 8;
  for (int64_t b = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); b < nb; b += stride) {
    const int64_t k = b * kBlock8;
    const int left = static_cast<int>(n - k < kBlock8 ? n - k : kBlock8);
    const bool w = vec && left == kBlock8;
    if (!ZS_CHECK(left > 0 && (!w || (aligned(m + k, 32) && aligned(v + k, 32) && aligned(q.exp_avg + k, 8) &&
                                      aligned(q.root + k, 8))),
                  81, k))
      continue;
    uint32_t cm[2], cr[2];
    load_codes(q.exp_avg + k, w, left, cm);
    load_codes(q.root + k, w, left, cr);
    float x[8], r[8];
    decode8(cm, q.exp_avg_scale[b], x);
    decode8(cr, q.root_scale[b], r);
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = __fmul_rn(r[j], r[j]);
    store_block_f32(m + k, w, left, x);
    store_block_f32(v + k, w, left, r);
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
