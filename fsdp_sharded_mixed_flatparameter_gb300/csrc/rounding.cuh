// rounding.cuh -- the hash behind stochastic rounding's draws, for the host
// (the launch's part: api.cu) and the device.  Internal.
#pragma once

#include <stdint.h>

#include "kernels.h"

namespace zs {

// The 32-bit PCG permutation (O'Neill, RXS-M-XS 32) as a hash.
__host__ __device__ __forceinline__ uint32_t pcg_hash(uint32_t x) {
  x = x * 747796405u + 2891336453u;
  x = ((x >> ((x >> 28) + 4u)) ^ x) * 277803737u;
  return (x >> 22) ^ x;
}

// Whether a moment needs 16 bits (its beta as the kernels have it, in binary32).
__host__ __device__ __forceinline__ bool exp_avg16(float beta1) {
  return beta1 > static_cast<float>(ZERO_EXP_AVG7_MAX_BETA1);
}
__host__ __device__ __forceinline__ bool root16(float beta2, int root_bits) {
  return root_bits == 16 || (root_bits == 0 && beta2 > static_cast<float>(ZERO_ROOT7_MAX_BETA2));
}

// The betas of a launch: with parameter groups the largest beta1, the least and
// the largest beta2; those that the launch does not know, as they are on the
// device, as here.
struct Betas {
  float beta1 = 1.0f, least2 = 0.0f, most2 = 1.0f;
};

// r: nullptr rounds to nearest.  step: nullptr when it will be read on the device.
inline RoundingBase rounding_base(const zero_rounding* r, const int64_t* step, const Betas& b) {
  if (r == nullptr) return RoundingBase{0u, 0u, kNearest, 0};
  uint32_t h = pcg_hash(static_cast<uint32_t>(r->seed));
  h = pcg_hash(static_cast<uint32_t>(r->seed >> 32) ^ h);
  if (step != nullptr) h = pcg_hash(static_cast<uint32_t>(*step) ^ h);
  const bool wide = root16(b.most2, r->root_bits);
  const int how = exp_avg16(b.beta1) || wide != root16(b.least2, r->root_bits) ? kByBeta : wide ? kRoot16 : kRoot7;
  return RoundingBase{h, static_cast<uint32_t>(r->stream), how, r->root_bits};
}

}  // namespace zs
