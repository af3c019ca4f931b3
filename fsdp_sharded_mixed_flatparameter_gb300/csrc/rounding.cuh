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

// Whether a root needs 16 bits (beta2 as the kernels have it, in binary32).
__host__ __device__ __forceinline__ bool root16(float beta2) {
  return beta2 > static_cast<float>(ZERO_ROOT7_MAX_BETA2);
}

// r: nullptr rounds to nearest.  step: nullptr when it will be read on the device.
// least, most: the step's beta2 (with parameter groups the least and the largest;
// 0 and 1 when the device has them).
inline RoundingBase rounding_base(const zero_rounding* r, const int64_t* step, float least, float most) {
  if (r == nullptr) return RoundingBase{0u, 0u, kNearest};
  uint32_t h = pcg_hash(static_cast<uint32_t>(r->seed));
  h = pcg_hash(static_cast<uint32_t>(r->seed >> 32) ^ h);
  if (step != nullptr) h = pcg_hash(static_cast<uint32_t>(*step) ^ h);
  int how = r->root_bits == 16 ? kRoot16 : kRoot7;
  if (r->root_bits == 0) how = root16(least) == root16(most) ? (root16(most) ? kRoot16 : kRoot7) : kRootBeta2;
  return RoundingBase{h, static_cast<uint32_t>(r->stream), how};
}

}  // namespace zs
