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

// r: nullptr rounds to nearest.  step: nullptr when it will be read on the device.
// beta2: the largest of the step's (0 when the device has them).
inline RoundingBase rounding_base(const zero_rounding* r, const int64_t* step, double beta2) {
  if (r == nullptr) return RoundingBase{0u, 0u, 0};
  uint32_t h = pcg_hash(static_cast<uint32_t>(r->seed));
  h = pcg_hash(static_cast<uint32_t>(r->seed >> 32) ^ h);
  if (step != nullptr) h = pcg_hash(static_cast<uint32_t>(*step) ^ h);
  const int bits = r->root_bits != 0 ? r->root_bits : beta2 > ZERO_ROOT7_MAX_BETA2 ? 16 : 7;
  return RoundingBase{h, static_cast<uint32_t>(r->stream), bits};
}

}  // namespace zs
