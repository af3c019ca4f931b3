// state8.cuh -- AdamW moments held in 8 bits: the format, its rounding and
// the per-element update.  Shared by the many-tensor step (adamw_list.cu),
// the flat-shard step (adamw_table8.cu) and the conversions (state8.cu).
// Internal; not part of the C ABI.
//
// The format.  A moment x is held as an e4m3 code c and one power of two S
// per block of 256 consecutive elements: x ~ c * S.  S is the least power of
// two (at least 2^-126) with max|x| <= 448 S over the block, 448 being the
// largest e4m3 value.  A power of two makes x / S and c * S exact, so the
// code's rounding is the only one; a floating code's relative error (at most
// 2^-4) does not depend on where S lies, only its lower end does: values
// below about 2^-14 of the block's largest lose bits, below 2^-18 vanish.
// S is kept as a binary32 number: 1/64 byte per element and moment.
//
// exp_avg_sq is held as its square root.  The root is what the update
// divides by, and computing it there anyway makes storing it free; its range
// inside a block (2^18) is a range of 2^36 for exp_avg_sq itself, whose
// elements differ by the squares of the grads' ratios.  A root above zero
// never becomes zero (codes below the smallest one are raised to it): a zero
// root under a surviving exp_avg would make the next update m / eps.
//
// Rounding to the code's grid is to nearest even, or stochastic: with u the
// grid's spacing at |x| / S and k a number in [0, 128) drawn for the element,
//   floor((floor(128 (|x| / S) / u) + k) / 128) u,
// whose mean is |x| / S to 1/128 of the spacing.  To nearest, a moment that
// moves by less than half a spacing per step (3 to 6 %; exp_avg_sq moves by
// 1 - beta2 of the difference) keeps its code until the block's S moves;
// stochastic rounding keeps the mean of the recurrence.  The draws are a
// hash of (seed, step, stream, element), so a step is reproducible.
#pragma once

#include "adam.cuh"
#include "common.cuh"

namespace zs {

constexpr int kBlock8 = 256;  // elements per scale: one warp, 8 elements per lane

// ------------------------------------------------------------------ codes
// 4 e4m3 codes (byte i = element i), widened exactly.
__device__ __forceinline__ void decode4(uint32_t c, float* x) {
  uint32_t a, b;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
      : "=r"(a), "=r"(b)
      : "r"(c));
  const float2 fa = __half22float2(*reinterpret_cast<const __half2*>(&a));
  const float2 fb = __half22float2(*reinterpret_cast<const __half2*>(&b));
  x[0] = fa.x;
  x[1] = fa.y;
  x[2] = fb.x;
  x[3] = fb.y;
}

// 4 values (|x| <= 448) to the nearest codes.
__device__ __forceinline__ uint32_t encode4_nearest(float x0, float x1, float x2, float x3) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\tmov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(x0), "f"(x1), "f"(x2), "f"(x3));
  return r;
}

// Two values, already scaled by 2^-8 (|x| <= 448 / 256), to codes in the low
// bytes of the result's halves.  binary16 has e4m3's exponents moved by 8
// (normal from 2^-14, below it spaced evenly) and 7 more fraction bits, so
// truncating to binary16 gives floor(128 |x| / u), adding the element's 7
// random bits (one per half of k) and dropping 7 gives the code.
__device__ __forceinline__ uint32_t encode2_stochastic(float x0, float x1, uint32_t k) {
  uint32_t h;
  asm("cvt.rz.f16x2.f32 %0, %2, %1;" : "=r"(h) : "f"(x0), "f"(x1));
  const uint32_t mag = (h & 0x7fff7fffu) + (k & 0x007f007fu);
  return ((mag >> 7) & 0x007f007fu) | ((h >> 8) & 0x00800080u);
}

// ------------------------------------------------------------------ scale
// (S, 1/S) of a block from the bits of max|x| (non-negative binary32 values
// order like their bits, NaN above all).  max|x| with a fraction above 1.75 =
// 448/256 needs the next power.  A block whose largest value is not finite,
// or 2^126 and more (where 1/S would leave the normal range), gets S = NaN:
// every element reads back as NaN.
__device__ __forceinline__ void block_scale(uint32_t amax, float& s, float& inv) {
  if (amax >= 0x7e800000u) {
    s = __uint_as_float(0x7fffffffu);
    inv = 0.0f;
    return;
  }
  const int e = max(static_cast<int>((amax + 0x1fffffu) >> 23) - 8, 1);
  s = __uint_as_float(static_cast<uint32_t>(e) << 23);
  inv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
}

// --------------------------------------------------------------- rounding
// The 32-bit PCG permutation (O'Neill, RXS-M-XS 32) as a hash.
__host__ __device__ __forceinline__ uint32_t pcg_hash(uint32_t x) {
  x = x * 747796405u + 2891336453u;
  x = ((x >> ((x >> 28) + 4u)) ^ x) * 277803737u;
  return (x >> 22) ^ x;
}

// The key of one block's draws: the word of pair i (elements 2i, 2i + 1) is
// pcg_hash(low 32 bits of i ^ key); of each half of it bits 0..6 round
// exp_avg and bits 7..13 the root.  `pair`: any pair of the block
// (a block never crosses a multiple of 2^32 pairs).
__device__ __forceinline__ uint32_t rounding_key(uint64_t seed, int64_t step, uint32_t stream, int64_t pair) {
  uint32_t h = pcg_hash(static_cast<uint32_t>(seed));
  h = pcg_hash(static_cast<uint32_t>(seed >> 32) ^ h);
  h = pcg_hash(static_cast<uint32_t>(step) ^ h);
  h = pcg_hash(stream ^ h);
  return pcg_hash(static_cast<uint32_t>(pair >> 32) ^ h);
}

// ----------------------------------------------------------------- update
// adam_update of adam.cuh on decoded moments: m, and r = sqrt(v) in place of
// v.  The moments' operations and roundings are the same; the denominator
// is sqrt(v) times fl(1 / sqrt(1 - beta2^t)) plus eps in one fma, where the
// 32-bit update divides: an IEEE division is about a dozen instructions,
// and with 16 instead of 30 bytes per element the update is near the issue
// limit, not only the bandwidth's.
__device__ __forceinline__ void adam_update8(float& p, float& m, float& r, float g, float coef, const AdamScalars& s,
                                             float inv_bc2_sqrt) {
  g = __fmul_rn(g, coef);
  p = __fmul_rn(p, s.decay);
  m = __fmaf_rn(s.omb1, g, __fmul_rn(m, s.b1));
  const float v = __fmaf_rn(__fmul_rn(s.omb2, g), g, __fmul_rn(__fmul_rn(r, r), s.b2));
  r = __fsqrt_rn(v);
  const float u = __fdiv_rn(m, __fmaf_rn(r, inv_bc2_sqrt, s.eps));
  p = __fsub_rn(p, __fmul_rn(s.step_size, u));
}

// ------------------------------------------------------------- one block
// A warp holds one block of 256 elements, 8 per lane: in vector order lane l
// has elements 8l .. 8l + 7, in element order l, l + 32, ..., l + 224 (tails
// and unaligned buffers; absent elements are zeros).
__device__ __forceinline__ int elem_of(bool vec, int lane, int j) { return vec ? 8 * lane + j : lane + 32 * j; }

__device__ __forceinline__ uint32_t warp_amax(const float (&x)[8]) {
  uint32_t a = 0u;
#pragma unroll
  for (int j = 0; j < 8; ++j) a = max(a, __float_as_uint(x[j]) & 0x7fffffffu);
  return __reduce_max_sync(0xffffffffu, a);
}

// Codes of the warp's block (c[0], c[1]: this lane's 8 elements, byte j of
// the pair = element j), and its scales.  Every lane must call it.
// `pair0`: the index of the block's first pair.
template <bool SR>
__device__ __forceinline__ void encode_block(const float (&m)[8], const float (&r)[8], bool vec, uint32_t key,
                                             int64_t pair0, uint32_t (&cm)[2], uint32_t (&cr)[2], float& sm,
                                             float& sr) {
  const int lane = threadIdx.x & 31;
  float im, ir;
  block_scale(warp_amax(m), sm, im);
  block_scale(warp_amax(r), sr, ir);
  if (SR) {  // 1/S >= 2^-118 in a finite block: 2^-8 of it is still normal
    im *= 0x1p-8f;
    ir *= 0x1p-8f;
  }
  const float least = SR ? 0x1p-17f : 0x1p-9f;  // the smallest code's value
  float x[8], y[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    x[j] = __fmul_rn(m[j], im);
    y[j] = __fmul_rn(r[j], ir);
    if (r[j] > 0.0f) y[j] = fmaxf(y[j], least);
  }
  if (!SR) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      cm[h] = encode4_nearest(x[4 * h], x[4 * h + 1], x[4 * h + 2], x[4 * h + 3]);
      cr[h] = encode4_nearest(y[4 * h], y[4 * h + 1], y[4 * h + 2], y[4 * h + 3]);
    }
  } else {
    uint32_t um[4], ur[4];
    const uint32_t p0 = static_cast<uint32_t>(pair0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w;
      if (vec) {
        w = pcg_hash((p0 + 4u * lane + i) ^ key);
      } else {  // elements lane + 64 i and lane + 64 i + 32: the same half of two words
        const uint32_t a = pcg_hash((p0 + 32u * i + (lane >> 1)) ^ key);
        const uint32_t b = pcg_hash((p0 + 32u * i + 16u + (lane >> 1)) ^ key);
        w = __byte_perm(a, b, (lane & 1) ? 0x7632 : 0x5410);
      }
      um[i] = encode2_stochastic(x[2 * i], x[2 * i + 1], w);
      ur[i] = encode2_stochastic(y[2 * i], y[2 * i + 1], w >> 7);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      cm[h] = __byte_perm(um[2 * h], um[2 * h + 1], 0x6420);
      cr[h] = __byte_perm(ur[2 * h], ur[2 * h + 1], 0x6420);
    }
  }
}

// 8 codes of one lane as floats.
__device__ __forceinline__ void decode8(const uint32_t (&c)[2], float s, float (&x)[8]) {
  decode4(c[0], x);
  decode4(c[1], x + 4);
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = __fmul_rn(x[j], s);
}

// This lane's codes of the block at `p` (its first element; `left` elements
// remain from there): one 8-byte load, or bytes in element order.
__device__ __forceinline__ void load_codes(const uint8_t* p, bool vec, int left, uint32_t (&c)[2]) {
  const int lane = threadIdx.x & 31;
  if (vec) {
    asm volatile("ld.global.cs.v2.u32 {%0,%1}, [%2];" : "=r"(c[0]), "=r"(c[1]) : "l"(p + 8 * lane));
  } else {
    c[0] = c[1] = 0u;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (lane + 32 * j < left) c[j >> 2] |= static_cast<uint32_t>(p[lane + 32 * j]) << (8 * (j & 3));
  }
}

__device__ __forceinline__ void store_codes(uint8_t* p, bool vec, int left, const uint32_t (&c)[2]) {
  const int lane = threadIdx.x & 31;
  if (vec) {
    asm volatile("st.global.cs.v2.u32 [%0], {%1,%2};" ::"l"(p + 8 * lane), "r"(c[0]), "r"(c[1]) : "memory");
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (lane + 32 * j < left) p[lane + 32 * j] = static_cast<uint8_t>(c[j >> 2] >> (8 * (j & 3)));
  }
}

// This lane's 8 binary32 values of a block, zeros beyond `left`.
__device__ __forceinline__ void load_block_f32(const float* p, bool vec, int left, float (&x)[8]) {
  const int lane = threadIdx.x & 31;
  if (vec) {
    ld8_rw(p + 8 * lane, x);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = (lane + 32 * j < left) ? p[lane + 32 * j] : 0.0f;
  }
}

__device__ __forceinline__ void store_block_f32(float* p, bool vec, int left, const float (&x)[8]) {
  const int lane = threadIdx.x & 31;
  if (vec) {
    st8(p + 8 * lane, x);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (lane + 32 * j < left) p[lane + 32 * j] = x[j];
  }
}

// The low-precision copy of a block's new parameters (lowp_dtype BF16 or
// F16; in vector order the address of each lane's 8 values is as aligned as
// the copy's start: 16, 8, 4 or 2 bytes).
__device__ __forceinline__ void store_block_lowp(void* lowp, int lowp_dtype, bool vec, int left,
                                                 const float (&x)[8]) {
  const int lane = threadIdx.x & 31;
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = (lowp_dtype == ZERO_BF16) ? pack2_rn<ZERO_BF16>(x[2 * i], x[2 * i + 1])
                                     : pack2_rn<ZERO_F16>(x[2 * i], x[2 * i + 1]);
  unsigned short* d = static_cast<unsigned short*>(lowp);
  if (vec && aligned(lowp, 16)) {
    st16(d + 8 * lane, make_uint4(w[0], w[1], w[2], w[3]));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = elem_of(vec, lane, j);
      if (vec || e < left) d[e] = static_cast<unsigned short>((j & 1) ? w[j >> 1] >> 16 : w[j >> 1] & 0xffffu);
    }
  }
}

}  // namespace zs
