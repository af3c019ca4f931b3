// adamw_table8.cu -- AdamW over one rank's flat shard with both moments in 8
// bits (state8.cuh), the grads read through the FlatParameter's tensor table
// (a flat grad is a table of one entry), optionally added to the earlier
// micro-batches' fp32 sum: the 8-bit counterpart of adamw_table_kernel.
// 16 instead of 28 bytes per parameter with 16-bit grads.
//
// Blocks of scales lie at shard elements 0, 256, ...: a block's warp owns
// one, a thread block 2048 consecutive elements.  The grads come as in
// adamw_table.cuh: directly, realigned in registers, or staged in shared
// memory where tensors meet.
#include "adam.cuh"
#include "common.cuh"
#include "kernels.h"
#include "state8.cuh"
#include "table.cuh"

namespace zs {

constexpr int kT8Block = 8 * kBlock8;

template <int DT, bool SR>
__global__ void __launch_bounds__(256)
    adamw_table8_kernel(float* __restrict__ p, zero_state8 q, const float* __restrict__ acc,
                        const zero_tensor* __restrict__ table, int n_tensors, int64_t shard_start, int64_t n,
                        float gscale, const float* __restrict__ dscale, void* __restrict__ lowp, int lowp_dtype,
                        bool state_vec, AdamScalars hs, const zero_adamw_device_state* __restrict__ ds, zero_rounding rnd,
                        int64_t step, const zero_norm_result* __restrict__ clip) {
  __shared__ float stage[kT8Block + kT8Block / 8];
  AdamScalars s = hs;
  if (ds != nullptr && !step_scalars<true>(hs, ds, s)) return;  // the prepared step is skipped
  if (dscale != nullptr) gscale = *dscale;
  float coef = 1.0f;
  if (clip != nullptr) {
    if (!clip->finite) return;  // non-finite grad norm: the step is skipped
    coef = clip->clip_coef;
  }
  constexpr int es = SrcTraits<DT>::esize;
  constexpr int vb = (DT == ZERO_F32) ? 32 : 16;
  const float inv = __frcp_rn(s.bc2_sqrt);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  bool unused_flag = false;  // the norm pass reports non-finite grads
  const int64_t nblk = (n + kT8Block - 1) / kT8Block;
  for (int64_t blk = blockIdx.x; blk < nblk; blk += gridDim.x) {
    const int64_t k0 = blk * kT8Block;
    const int blen = static_cast<int>(n - k0 < kT8Block ? n - k0 : kT8Block);
    const int64_t k = k0 + kBlock8 * warp;
    const int left = static_cast<int>(n - k < kBlock8 ? n - k : kBlock8);  // <= 0: nothing for this warp
    const bool vec = state_vec && left == kBlock8;
    const int64_t b = k / kBlock8;
    if (!ZS_CHECK(!vec || (k + kBlock8 <= n && aligned(p + k, 32) && aligned(q.exp_avg + k, 8) &&
                           aligned(q.root + k, 8) && (acc == nullptr || aligned(acc + k, 32))),
                  70, k))
      return;
    float pr[8], ar[8];
    uint32_t cm[2], cr[2];
    float sm = 0.0f, sr = 0.0f;
    if (left > 0) {
      load_block_f32(p + k, vec, left, pr);
      load_codes(q.exp_avg + k, vec, left, cm);
      load_codes(q.root + k, vec, left, cr);
      sm = q.exp_avg_scale[b];
      sr = q.root_scale[b];
      if (acc != nullptr) load_block_f32(acc + k, vec, left, ar);
    }
    const int64_t f0 = shard_start + k0;
    const int ti = find_tensor_warp(table, n_tensors, f0);
    const void* tptr = table[ti].ptr;
    const int64_t toff = __ldg(&table[ti].flat_offset), tnum = __ldg(&table[ti].numel);
    const char* tsrc = tptr ? static_cast<const char*>(tptr) + es * (f0 - toff) : nullptr;
    const bool inside = state_vec && blen == kT8Block && tsrc != nullptr && toff <= f0 && f0 + kT8Block <= toff + tnum;
    const bool direct = inside && reinterpret_cast<uintptr_t>(tsrc) % vb == 0;
    const bool shifted = DT != ZERO_F32 && inside && !direct && f0 - toff >= 8 && f0 + kT8Block + 8 <= toff + tnum &&
                         ZS_CHECK(aligned(tsrc, es), 73, k);
    float g[8];
    if (direct) {
      load8_src<DT>(tsrc + es * 8 * threadIdx.x, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = __fmul_rn(gscale, g[j]);
    } else if (shifted) {
      float xs[1][8];
      load8_shifted<DT, 1>(tsrc, xs);
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = __fmul_rn(gscale, xs[0][j]);
    } else {
      stage_range<DT>(table, n_tensors, ti, f0, f0 + blen, gscale, stage, unused_flag);
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e = elem_of(vec, lane, j);
        g[j] = (vec || e < left) ? stage[stage_idx(kBlock8 * warp + e)] : 0.0f;
      }
      __syncthreads();
    }
    if (left <= 0) continue;
    if (acc != nullptr) {
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = __fadd_rn(ar[j], g[j]);
    }
    float m[8], r[8];
    decode8(cm, sm, m);
    decode8(cr, sr, r);
#pragma unroll
    for (int j = 0; j < 8; ++j) adam_update8(pr[j], m[j], r[j], g[j], coef, s, inv);
    uint32_t key = 0u;
    if (SR)
      key = rounding_key(rnd.seed, ds != nullptr ? ds->step : step, static_cast<uint32_t>(rnd.stream), k >> 1);
    encode_block<SR>(m, r, vec, key, k >> 1, cm, cr, sm, sr);
    store_block_f32(p + k, vec, left, pr);
    store_codes(q.exp_avg + k, vec, left, cm);
    store_codes(q.root + k, vec, left, cr);
    if (lane == 0) {
      q.exp_avg_scale[b] = sm;
      q.root_scale[b] = sr;
    }
    if (lowp != nullptr) store_block_lowp(static_cast<unsigned short*>(lowp) + k, lowp_dtype, vec, left, pr);
  }
}

template <int DT>
static zero_status launch_table8_dt(const Table8Args& a, const AdamScalars& s, cudaStream_t st) {
  const bool sv = aligned(a.p, 32) && aligned(a.q.exp_avg, 8) && aligned(a.q.root, 8) &&
                  (a.acc == nullptr || aligned(a.acc, 32));
  const unsigned grid = one_pass_blocks(a.n, kT8Block);
  if (a.stochastic)
    adamw_table8_kernel<DT, true><<<grid, 256, 0, st>>>(a.p, a.q, a.acc, a.table, a.n_tensors, a.shard_start, a.n,
                                                        a.gscale, a.dscale, a.lowp, a.lowp_dtype, sv, s, a.ds, a.rounding,
                                                        a.step, a.clip);
  else
    adamw_table8_kernel<DT, false><<<grid, 256, 0, st>>>(a.p, a.q, a.acc, a.table, a.n_tensors, a.shard_start, a.n,
                                                         a.gscale, a.dscale, a.lowp, a.lowp_dtype, sv, s, a.ds,
                                                         a.rounding, a.step, a.clip);
  return check_launch("adamw_table8_kernel");
}

ZS_DEBUG_UNIT(adamw_table8)

zero_status launch_adamw_table8(const Table8Args& a, const AdamScalars& s, cudaStream_t st) {
  if (a.grad_dtype == ZERO_F32) return launch_table8_dt<ZERO_F32>(a, s, st);
  if (a.grad_dtype == ZERO_BF16) return launch_table8_dt<ZERO_BF16>(a, s, st);
  return launch_table8_dt<ZERO_F16>(a, s, st);
}

}  // namespace zs
