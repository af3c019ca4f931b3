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
// grid's spacing at |x| / S,
//   7 bits:  floor((floor(128 (|x| / S) / u) + k) / 128) u,  k in [0, 128) drawn,
//   16 bits: floor((|x| / S) / u + (h + 1/2) / 65536) u,  h in [0, 65536) drawn.
// The 16 bits keep the mean to 2^-17 u, whatever x.  The 7 bits are u / 256 low
// on average and do not see a move of less than u / 128, which a recurrence
// adds up over 1 / (1 - beta) steps: exp_avg comes to 0.99 of what it should be
// at beta1 = 0.95, 0.96 at 0.99 and 0.75 at 0.999; exp_avg_sq, normal grads, 8000 steps from zero, comes to
// 0.68 of what it should be at beta2 = 0.999 and 0.24 at 0.9999 (with the 16
// bits to 1.04 and 1.03: the square of the root's own noise).  exp_avg takes
// the 16 from beta1 > 0.95 on (ZERO_EXP_AVG7_MAX_BETA1), the root from beta2 >
// 0.99 on (ZERO_ROOT7_MAX_BETA2), up to which the 7 bits stay as near (0.97 at 0.99, 1.01 at 0.95; 16 bits 1.04,
// 1.03) in 4 instructions an element less (1.88e9 elements: 4.53 against 4.58
// ms; a flat shard of 1.63e9: 3.89 against 3.96).  To nearest, a moment that
// moves by less than half a spacing per step (3 to 6 %) keeps its code until
// the block's S moves: the same exp_avg_sq comes to 4.9 at beta2 = 0.95, to
// 0.19 at 0.999.  The draws are a hash of (seed, step, stream, element), so a
// step is reproducible.
#pragma once

#include "adam.cuh"
#include "common.cuh"
#include "rounding.cuh"

namespace zs {

constexpr int kBlock8 = 256;  // elements per scale: one warp, 8 elements per lane

// ------------------------------------------------------------------ pairs
// Two binary32 values in one 64-bit register pair: sm_100's packed
// arithmetic does both in one instruction, each rounded as alone.  The update
// is bound by instructions before it is bound by the arithmetic units, so
// everything that can be is done in pairs.
using F2 = unsigned long long;

__device__ __forceinline__ F2 pair(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ F2 both(float a) { return pair(a, a); }
__device__ __forceinline__ void unpair(F2 x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Hardware reciprocal and reciprocal root (relative error under 2^-22,
// subnormal arguments and results as zero).
__device__ __forceinline__ float reciprocal_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rsqrt_approx(float x) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// sqrt(v) of finite v >= 0: g = v y with y ~ 1 / sqrt(v), then one Newton step
// g + (v - g^2) y / 2, whose residual is exact in an fma.  Its error before the
// last rounding is of the order of y's squared, so from any y within 2^-22 it is
// the correctly rounded root but for a v in a million or two (1 ulp off there);
// from this GPU's y it is the correctly rounded one for all 2^24 values of
// [1, 4).  Zero gives zero; below the normal range (2^-126) it is positive but
// too small (kLift).
__device__ __forceinline__ F2 root2(F2 v) {
  float v0, v1;
  unpair(v, v0, v1);
  const F2 y = pair(rsqrt_approx(fmaxf(v0, 0x1p-126f)), rsqrt_approx(fmaxf(v1, 0x1p-126f)));
  const F2 g = mul2(v, y);
  return fma2(fma2(g, g, mul2(v, both(-1.0f))), mul2(y, both(-0.5f)), g);
}

// ------------------------------------------------------------------ codes
// 4 e4m3 codes (byte i = element i) as two pairs, widened exactly.
__device__ __forceinline__ void decode4(uint32_t c, F2& a, F2& b) {
  uint32_t lo, hi;
  asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\tcvt.rn.f16x2.e4m3x2 %1, y;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(c));
  const float2 fa = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 fb = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  a = pair(fa.x, fa.y);
  b = pair(fb.x, fb.y);
}

// 4 values (|x| <= 448) to the nearest codes.
__device__ __forceinline__ uint32_t encode4_nearest(F2 a, F2 b) {
  float x0, x1, x2, x3;
  unpair(a, x0, x1);
  unpair(b, x2, x3);
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\tmov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(x0), "f"(x1), "f"(x2), "f"(x3));
  return r;
}

// 4 values, already scaled by 2^-8 (|x| <= 448 / 256), to codes by stochastic
// rounding; k0, k1: twice the elements' 7-bit numbers, in the halves of a word
// for each pair.  binary16 has e4m3's exponents moved by 8 (normal from
// 2^-14, below it spaced evenly) and 7 more fraction bits: truncated to
// binary16 a value is floor(128 |x| / u), adding the number carries into the
// code, and doubled (the sign bit is taken out, |x| < 2 leaves bit 14 free)
// the code fills the upper byte of each half, where one byte permutation
// collects four.
template <bool SIGNED>
__device__ __forceinline__ uint32_t encode4_stochastic(F2 a, F2 b, uint32_t k0, uint32_t k1) {
  float x0, x1, x2, x3;
  unpair(a, x0, x1);
  unpair(b, x2, x3);
  uint32_t h0, h1;
  asm("cvt.rz.f16x2.f32 %0, %2, %1;" : "=r"(h0) : "f"(x0), "f"(x1));
  asm("cvt.rz.f16x2.f32 %0, %2, %1;" : "=r"(h1) : "f"(x2), "f"(x3));
  if (!SIGNED) return __byte_perm(2u * h0 + k0, 2u * h1 + k1, 0x7531);
  const uint32_t c = __byte_perm(2u * (h0 & 0x7fff7fffu) + k0, 2u * (h1 & 0x7fff7fffu) + k1, 0x7531);
  return c | (__byte_perm(h0, h1, 0x7531) & 0x80808080u);
}

// 4 roots, already scaled by 2^-24 (0 <= y <= 448 2^-24 but for an ulp), to
// codes by stochastic rounding with 16 bits each: w0, w1 hold the numbers h in
// their halves.  From 2^-6 (here 2^-30) on the upper 12 bits of a binary32
// value are its e4m3 code but for the exponent, which the scale has moved to
// 96 + e: in the word's bits 20 .. 27 stands e, then the fraction.  Four bits
// further up the code is the upper byte and (h + 1/2) / 65536 of its unit is
// added as the bytes 00 h h 80.  Below 2^-6 the grid is even: y / 2 + 2^-31 has
// exponent 96, e = 0, and a fraction of the same units.  y above its limit by
// an ulp (2^-20 u) cannot carry into the NaN code: h + 1/2 leaves 2^-17 u.
// SIGNED (exp_avg): the same of |y|, under y's sign, with h's bytes exchanged, so
// that the two moments' roundings do not go together.
template <bool SIGNED>
__device__ __forceinline__ uint32_t encode4_16(F2 a, F2 b, uint32_t w0, uint32_t w1) {
  float y[4];
  unpair(a, y[0], y[1]);
  unpair(b, y[2], y[3]);
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float z = fabsf(y[i]) < 0x1p-30f ? fmaf(fabsf(y[i]), 0.5f, 0x1p-31f) : y[i];
    const uint32_t h = __byte_perm(i < 2 ? w0 : w1, 0x80u,
                                   SIGNED ? ((i & 1) ? 0x5234 : 0x5014) : ((i & 1) ? 0x5324 : 0x5104));
    c[i] = (__float_as_uint(z) << 4) + h;  // the sign leaves
  }
  const uint32_t code = __byte_perm(__byte_perm(c[0], c[1], 0x0073), __byte_perm(c[2], c[3], 0x0073), 0x5410);
  if (!SIGNED) return code;
  const uint32_t s0 = __byte_perm(__float_as_uint(y[0]), __float_as_uint(y[1]), 0x0073);
  const uint32_t s1 = __byte_perm(__float_as_uint(y[2]), __float_as_uint(y[3]), 0x0073);
  return code | (__byte_perm(s0, s1, 0x5410) & 0x80808080u);
}

// ------------------------------------------------------------------ scale
// (S, 1/S) of a block from the bits of max|x| (non-negative binary32 values
// order like their bits, NaN above all).  max|x| with a fraction above 1.75 =
// 448/256 needs the next power.  A block whose largest value is not finite,
// or 2^126 and more (where 1/S would leave the normal range), gets S = NaN:
// every element reads back as NaN.  `least`: the exponent field of the least S.
__device__ __forceinline__ void block_scale(uint32_t amax, int least, float& s, float& inv) {
  if (amax >= 0x7e800000u) {
    s = __uint_as_float(0x7fffffffu);
    inv = 0.0f;
    return;
  }
  const int e = max(static_cast<int>((amax + 0x1fffffu) >> 23) - 8, least);
  s = __uint_as_float(static_cast<uint32_t>(e) << 23);
  inv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
}

// --------------------------------------------------------------- rounding
// The key of one block's draws (pcg_hash: rounding.cuh): the word of pair i
// (elements 2i, 2i + 1) is pcg_hash(low 32 bits of i ^ key); of each half of it
// bits 0..6, or all 16, round exp_avg and bits 7..13, or all 16, the root (the
// two moments' roundings then share bits, which their means do not see).  The launch has hashed the
// seed and the step; a step on the device (ds) is hashed here.  `pair`: any
// pair of the block (a block never crosses a multiple of 2^32 pairs).
__device__ __forceinline__ uint32_t rounding_key(const RoundingBase& rnd, const zero_adamw_device_state* ds,
                                                 uint32_t tensor, int64_t pair) {
  uint32_t h = rnd.hash;
  if (ds != nullptr) h = pcg_hash(static_cast<uint32_t>(ds->step) ^ h);
  h = pcg_hash((rnd.stream + tensor) ^ h);
  return pcg_hash(static_cast<uint32_t>(pair >> 32) ^ h);
}

// ----------------------------------------------------------------- update
// Blocks of small roots are computed 2^40 times larger: v as 2^80 v, its factors
// lifted (powers of two: no other rounding), and r's factor and its scale take
// 2^-40.  Else S^2 beta2 would be zero from S = 2^-75 on, where v is not yet, and
// root2 is too small for a v under 2^-126.  A block needs it where S^2 beta2 <
// 2^-100: from there up a new v under 2^-126 has a root under 2^-10 of the new S
// and is raised to the smallest code, whatever root2 gives; its r itself, under
// 2^-63, is lost in eps unless eps is under 2^-34, and then every block needs it.
// A block that could overflow by it (grads of 2^20 and more, S of 2^14 and more
// unless beta2 is 0) is left as it is.
constexpr float kLift = 0x1p40f;
constexpr int kLiftLog2 = 40;

__device__ __forceinline__ uint32_t warp_amax(const F2 (&x)[4]);

__device__ __forceinline__ bool small_roots(const AdamScalars& s, float sr) {
  return __fmul_rn(__fmul_rn(sr, sr), s.b2) < 0x1p-100f || s.eps < 0x1p-34f;
}

__device__ __forceinline__ bool liftable(const AdamScalars& s, float sr, const float (&g)[8], float coef) {
  const F2 x[4] = {pair(g[0], g[1]), pair(g[2], g[3]), pair(g[4], g[5]), pair(g[6], g[7])};
  return __fmul_rn(__uint_as_float(warp_amax(x)), fabsf(coef)) < 0x1p20f && (sr < 0x1p14f || s.b2 == 0.0f);
}

// The update's factors for one block, each twice.  The decoded moments enter
// only as m beta1 = c (S beta1) and v beta2 = c^2 (S^2 beta2), which with S a
// power of two are the same numbers as fl(m beta1) and fl(fl(r^2) beta2), as
// these factors and r^2 are normal numbers (kLift; S beta1 loses a bit or two in
// blocks of S = 2^-126).
struct Factors8 {
  F2 coef, decay, mb1, omb1, vb2, omb2, inv_bc2, eps, step;
};

__device__ __forceinline__ Factors8 factors8(const AdamScalars& s, float sm, float sr, float coef, bool lift) {
  Factors8 f;
  if (lift) sr = fminf(__fmul_rn(sr, kLift), 0x1p54f);  // larger only where beta2 is 0
  f.coef = both(coef);
  f.decay = both(s.decay);
  f.mb1 = both(__fmul_rn(sm, s.b1));
  f.omb1 = both(s.omb1);
  f.vb2 = both(__fmul_rn(__fmul_rn(sr, sr), s.b2));
  f.omb2 = both(lift ? __fmul_rn(s.omb2, kLift * kLift) : s.omb2);
  const float inv_bc2 = __frcp_rn(s.bc2_sqrt);
  f.inv_bc2 = both(lift ? __fmul_rn(inv_bc2, 1.0f / kLift) : inv_bc2);
  f.eps = both(fmaxf(s.eps, 0x1p-126f));  // the reciprocal's argument stays normal
  f.step = both(-s.step_size);
  return f;
}

// The 32-bit update (adam.cuh) on two elements, in two parts.  First the
// moments, from codes: cm, cr (the codes' values) in, m and v (lifted: 2^80 v) out,
// bit for bit what the 32-bit update gives for the decoded moments where it has
// 24 bits for them.
__device__ __forceinline__ void moments8(F2& cm, F2& cr, F2 g, const Factors8& f) {
  g = mul2(g, f.coef);
  cm = fma2(f.omb1, g, mul2(cm, f.mb1));
  cr = fma2(mul2(f.omb2, g), g, mul2(mul2(cr, cr), f.vb2));
}

// Then the parameter: p - step m / (r / sqrt(1 - beta2^t) + eps), r = sqrt(v),
// with the hardware's reciprocal, its change within 8 ulp of itself: correctly
// rounded division and root by the compiler's sequences are some 25
// instructions and two branches an element, together as much as all the rest.
__device__ __forceinline__ F2 param8(F2 p, F2 m, F2 r, const Factors8& f) {
  float d0, d1;
  unpair(fma2(r, f.inv_bc2, f.eps), d0, d1);
  const F2 u = mul2(m, pair(reciprocal_approx(d0), reciprocal_approx(d1)));
  return fma2(f.step, u, mul2(p, f.decay));
}

// ------------------------------------------------------------- one block
// A warp holds one block of 256 elements, 8 per lane.  VEC: lane l has
// elements 8l .. 8l + 7 of a full block in aligned buffers; else it has
// elements l, l + 32, ..., l + 224, those from `left` on absent (zeros): tails
// and unaligned buffers.  The two are separate instantiations: one code for
// both, with the order as a variable, took 100 registers (adamw_list8.cu).
template <bool VEC>
__device__ __forceinline__ int elem_of(int j) {
  const int lane = threadIdx.x & 31;
  return VEC ? 8 * lane + j : lane + 32 * j;
}

// max|x| over the warp's block, as bits (NaN is the largest).
__device__ __forceinline__ uint32_t warp_amax(const F2 (&x)[4]) {
  float a = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float x0, x1;
    unpair(x[i], x0, x1);
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(a) : "f"(a), "f"(x0), "f"(x1));
  }
  return __reduce_max_sync(0xffffffffu, __float_as_uint(a));
}

// Codes of the warp's block (byte j of the pair = this lane's element j) and
// its scales, from m, r = sqrt(v) and the block's max|m|, max r as bits.
// Every lane must call it.  `pair0`: the block's first pair; lift: r is kLift times
// the root; wide_m, wide_r: 16 bits (SR == kByBeta).
template <bool VEC, int SR>
__device__ __forceinline__ void encode_block(const F2 (&m)[4], const F2 (&r)[4], uint32_t amax_m, uint32_t amax_r,
                                             uint32_t key, int64_t pair0, uint2& cm, uint2& cr, float& sm,
                                             float& sr, bool lift, bool wide_m, bool wide_r) {
  float im, ir;
  block_scale(amax_m, 1, sm, im);
  block_scale(amax_r, lift ? 1 + kLiftLog2 : 1, sr, ir);
  if (lift) sr *= 1.0f / kLift;
  if (SR != kByBeta) wide_m = false, wide_r = SR == kRoot16;
  // 1/S >= 2^-118 in a finite block: 2^-24 of it is not normal any more, but exact
  im *= SR == kNearest ? 1.0f : wide_m ? 0x1p-24f : 0x1p-8f;
  const float to = SR == kNearest ? 1.0f : wide_r ? 0x1p-24f : 0x1p-8f;
  ir *= to;  // a root is at most 2^64, 1/S at least 2^-56
  const float least = 0x1p-9f * to;  // the smallest code's value
  F2 x[4], y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = mul2(m[i], both(im));
    y[i] = mul2(r[i], both(ir));
    float y0, y1, r0, r1;
    unpair(y[i], y0, y1);
    unpair(r[i], r0, r1);
    if (r0 > 0.0f) y0 = fmaxf(y0, least);
    if (r1 > 0.0f) y1 = fmaxf(y1, least);
    y[i] = pair(y0, y1);
  }
  if (SR == kNearest) {
    cm = make_uint2(encode4_nearest(x[0], x[1]), encode4_nearest(x[2], x[3]));
    cr = make_uint2(encode4_nearest(y[0], y[1]), encode4_nearest(y[2], y[3]));
  } else {
    const int lane = threadIdx.x & 31;
    uint32_t km[4], wr[4];
    const uint32_t p0 = static_cast<uint32_t>(pair0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w;
      if (VEC) {
        w = pcg_hash((p0 + 4u * lane + i) ^ key);
      } else {  // elements lane + 64 i and lane + 64 i + 32: the same half of two words
        const uint32_t a = pcg_hash((p0 + 32u * i + (lane >> 1)) ^ key);
        const uint32_t b = pcg_hash((p0 + 32u * i + 16u + (lane >> 1)) ^ key);
        w = __byte_perm(a, b, (lane & 1) ? 0x7632 : 0x5410);
      }
      km[i] = (w << 1) & 0x00fe00feu;
      wr[i] = w;
    }
    if (wide_m)
      cm = make_uint2(encode4_16<true>(x[0], x[1], wr[0], wr[1]), encode4_16<true>(x[2], x[3], wr[2], wr[3]));
    else
      cm = make_uint2(encode4_stochastic<true>(x[0], x[1], km[0], km[1]),
                      encode4_stochastic<true>(x[2], x[3], km[2], km[3]));
    if (wide_r) {
      cr = make_uint2(encode4_16<false>(y[0], y[1], wr[0], wr[1]), encode4_16<false>(y[2], y[3], wr[2], wr[3]));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) wr[i] = (wr[i] >> 6) & 0x00fe00feu;
      cr = make_uint2(encode4_stochastic<false>(y[0], y[1], wr[0], wr[1]),
                      encode4_stochastic<false>(y[2], y[3], wr[2], wr[3]));
    }
  }
}

// The values of one lane's 8 codes.
__device__ __forceinline__ void decode8(uint2 c, F2 (&x)[4]) {
  decode4(c.x, x[0], x[1]);
  decode4(c.y, x[2], x[3]);
}

// This lane's codes of the block that starts at `p`.
template <bool VEC>
__device__ __forceinline__ uint2 load_codes(const uint8_t* p, int left) {
  uint2 c = make_uint2(0u, 0u);
  if (VEC) {
    asm volatile("ld.global.cs.v2.u32 {%0,%1}, [%2];" : "=r"(c.x), "=r"(c.y) : "l"(p + elem_of<VEC>(0)));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (elem_of<VEC>(j) < left) (j < 4 ? c.x : c.y) |= static_cast<uint32_t>(p[elem_of<VEC>(j)]) << (8 * (j & 3));
  }
  return c;
}

template <bool VEC>
__device__ __forceinline__ void store_codes(uint8_t* p, int left, uint2 c) {
  if (VEC) {
    asm volatile("st.global.cs.v2.u32 [%0], {%1,%2};" ::"l"(p + elem_of<VEC>(0)), "r"(c.x), "r"(c.y) : "memory");
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (elem_of<VEC>(j) < left) p[elem_of<VEC>(j)] = static_cast<uint8_t>((j < 4 ? c.x : c.y) >> (8 * (j & 3)));
  }
}

// This lane's 8 binary32 values of the block that starts at `p`.
template <bool VEC>
__device__ __forceinline__ void load_block_f32(const float* p, int left, float (&x)[8]) {
  if (VEC) {
    ld8_rw(p + elem_of<VEC>(0), x);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = (elem_of<VEC>(j) < left) ? p[elem_of<VEC>(j)] : 0.0f;
  }
}

template <bool VEC>
__device__ __forceinline__ void store_block_f32(float* p, int left, const float (&x)[8]) {
  if (VEC) {
    st8(p + elem_of<VEC>(0), x);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (elem_of<VEC>(j) < left) p[elem_of<VEC>(j)] = x[j];
  }
}

// The low-precision copy of a block's new parameters (BF16 or F16, at any
// 2-byte alignment).
template <bool VEC>
__device__ __forceinline__ void store_block_lowp(void* lowp, int lowp_dtype, int left, const float (&x)[8]) {
  uint32_t w[4];
  if (lowp_dtype == ZERO_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack2_rn<ZERO_BF16>(x[2 * i], x[2 * i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack2_rn<ZERO_F16>(x[2 * i], x[2 * i + 1]);
  }
  unsigned short* d = static_cast<unsigned short*>(lowp);
  if (VEC && aligned(lowp, 16)) {
    st16(d + elem_of<VEC>(0), make_uint4(w[0], w[1], w[2], w[3]));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (VEC || elem_of<VEC>(j) < left)
        d[elem_of<VEC>(j)] = static_cast<unsigned short>((j & 1) ? w[j >> 1] >> 16 : w[j >> 1] & 0xffffu);
  }
}

// The update of one block whose codes, scales and grads (fl(scale x), summed)
// are in registers, and its stores.  ROOTS: what is known of the block's
// small_roots().
enum Roots : int { kLarge, kSmall, kAnyRoots };

template <bool VEC, int SR, int ROOTS>
__device__ __forceinline__ void update_block(float* p, uint8_t* qm, uint8_t* qr, float* ms, float* rs,
                                             unsigned short* lowp, int lowp_dtype, int left, const float (&x)[8],
                                             const float (&g)[8], uint2 cm, uint2 cr, float sm, float sr, float coef,
                                             const AdamScalars& s, uint32_t key, int root_bits, int64_t pair0) {
  const bool lift = ROOTS != kLarge && (ROOTS == kSmall || small_roots(s, sr)) && liftable(s, sr, g, coef);
  const Factors8 f = factors8(s, sm, sr, coef, lift);
  F2 m[4], r[4];
  float y[8];
  decode8(cm, m);
  decode8(cr, r);
#pragma unroll
  for (int i = 0; i < 4; ++i) moments8(m[i], r[i], pair(g[2 * i], g[2 * i + 1]), f);
  const uint32_t amax_m = warp_amax(m), amax_v = warp_amax(r);
  if (amax_v < 0x7f800000u) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = root2(r[i]);
  } else {  // an overflown or NaN exp_avg_sq in the block: the same, for any value
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v0, v1;
      unpair(r[i], v0, v1);
      r[i] = pair(__fsqrt_rn(v0), __fsqrt_rn(v1));
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) unpair(param8(pair(x[2 * i], x[2 * i + 1]), m[i], r[i], f), y[2 * i], y[2 * i + 1]);
  store_block_f32<VEC>(p, left, y);
  if (lowp != nullptr) store_block_lowp<VEC>(lowp, lowp_dtype, left, y);
  // the largest root is the root of the largest exp_avg_sq
  encode_block<VEC, SR>(m, r, amax_m, __float_as_uint(__fsqrt_rn(__uint_as_float(amax_v))), key, pair0, cm, cr, sm, sr,
                        lift, exp_avg16(s.b1), root16(s.b2, root_bits));
  store_codes<VEC>(qm, left, cm);
  store_codes<VEC>(qr, left, cr);
  if ((threadIdx.x & 31) == 0) {
    *ms = sm;
    *rs = sr;
  }
}

// The same for any block with the two cases apart: in the flat-shard kernel one
// code for both spilled (1.63e9 elements: 4.20 against 3.72 ms); in the list's,
// two did (1.88e9, stochastic: 4.59 against 4.50).
template <bool VEC, int SR>
__device__ __forceinline__ void update_block_split(float* p, uint8_t* qm, uint8_t* qr, float* ms, float* rs,
                                                   unsigned short* lowp, int lowp_dtype, int left, const float (&x)[8],
                                                   const float (&g)[8], uint2 cm, uint2 cr, float sm, float sr, float coef,
                                                   const AdamScalars& s, uint32_t key, int root_bits, int64_t pair0) {
  if (small_roots(s, sr))
    update_block<VEC, SR, kSmall>(p, qm, qr, ms, rs, lowp, lowp_dtype, left, x, g, cm, cr, sm, sr, coef, s, key,
                                 root_bits, pair0);
  else
    update_block<VEC, SR, kLarge>(p, qm, qr, ms, rs, lowp, lowp_dtype, left, x, g, cm, cr, sm, sr, coef, s, key,
                                 root_bits, pair0);
}

}  // namespace zs
