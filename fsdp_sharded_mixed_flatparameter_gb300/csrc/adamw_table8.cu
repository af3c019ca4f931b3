// adamw_table8.cu -- AdamW over one rank's flat shard with both moments in 8
// bits (state8.cuh), the grads read through the FlatParameter's tensor table
// (a flat grad is a table of one entry), optionally added to the earlier
// micro-batches' fp32 sum: the 8-bit counterpart of adamw_table_kernel.
// 16 instead of 28 bytes per parameter with 16-bit grads.
//
// Blocks of scales lie at shard elements 0, 256, ...: a block's warp owns
// one, a thread block 2048 consecutive elements.  The grads come as in
// adamw_table.cuh: directly, realigned in registers (fp32: in shared memory, a
// warp alone), or staged in shared memory by the block where tensors meet.
//
// Measured: a Llama-13B ZeRO-3 shard (1.63e9 elements, flat fp16 grads) 3.72
// ms = 7.03 TB/s; a quarter of 20,000 ragged tensors (377e6, most parts off
// the 16-byte grid, stochastic) 1.03 ms = 5.88 TB/s, 81 instructions an
// element with the search and the realignment; a GPT-2 ZeRO-1 shard with
// accumulation (15.6e6) 53 us = 5.85 TB/s, ten waves of blocks.  Five
// blocks per SM (48 registers) against four: 3.71 and 1.09 against 3.88 and
// 1.19 ms; six spill.  Two or four parts per block and search: 1.40 and 1.32
// ms (ragged); blocks of 128 threads: the same; one warp's search shared
// through a barrier: 1.04.
#include "adam.cuh"
#include "common.cuh"
#include "kernels.h"
#include "state8.cuh"
#include "table.cuh"

namespace zs {

constexpr int kT8Block = 8 * kBlock8;

// A full part (2048 elements, state and accumulator aligned).  The search of
// the table comes before the state's loads, although those do not depend on
// it: its three rounds of short reads then do not queue behind them (20,000
// ragged tensors, 377M elements: 998 against 1040 us).  Every thread of the
// block must call it.
template <int DT, int SR>
__device__ __forceinline__ void table8_full(float* p, const zero_state8& q, const float* acc, const zero_tensor* table,
                                            int n_tensors, int64_t shard_start, int64_t k0, float gscale, void* lowp,
                                            int lowp_dtype, float coef, const AdamScalars& s, uint32_t key,
                                            int root_bits, float* stage) {
  constexpr int es = SrcTraits<DT>::esize;
  constexpr int vb = (DT == ZERO_F32) ? 32 : 16;
  const int warp = threadIdx.x >> 5;
  const int64_t k = k0 + kBlock8 * warp, b = k / kBlock8, f0 = shard_start + k0;
  float pr[8], g[8];
  const int ti = find_tensor_warp(table, n_tensors, f0);
  load_block_f32<true>(p + k, kBlock8, pr);
  const uint2 cm = load_codes<true>(q.exp_avg + k, kBlock8), cr = load_codes<true>(q.root + k, kBlock8);
  const float sm = q.exp_avg_scale[b], sr = q.root_scale[b];
  const void* tptr = table[ti].ptr;
  const int64_t toff = __ldg(&table[ti].flat_offset), tnum = __ldg(&table[ti].numel);
  const char* tsrc = tptr ? static_cast<const char*>(tptr) + es * (f0 - toff) : nullptr;
  const bool inside = tsrc != nullptr && toff <= f0 && f0 + kT8Block <= toff + tnum;
  const bool direct = inside && reinterpret_cast<uintptr_t>(tsrc) % vb == 0;
  const bool shifted = DT != ZERO_F32 && inside && !direct && f0 - toff >= 8 && f0 + kT8Block + 8 <= toff + tnum &&
                       ZS_CHECK(aligned(tsrc, es), 73, k);
  if (direct) {
    load8_src<DT>(tsrc + es * 8 * threadIdx.x, g);
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = __fmul_rn(gscale, g[j]);
  } else if (shifted) {
    float xs[1][8];
    load8_shifted<DT, 1>(tsrc, xs);
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = __fmul_rn(gscale, xs[0][j]);
  } else if (DT == ZERO_F32 && inside) {
    // binary32 grads off the 32-byte grid: each warp reads its 256 in order and turns them in shared memory, alone
    // (through the block's stage, as where tensors meet: 1.32 against 1.13 ms for 20,000 ragged fp32 tensors, 377e6)
    float* const turn = stage + (kBlock8 + kBlock8 / 8) * warp;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      turn[stage_idx(lane + 32 * j)] = __fmul_rn(gscale, load_elem<DT>(tsrc, kBlock8 * warp + lane + 32 * j));
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = turn[stage_idx(8 * lane + j)];
  } else {
    bool unused_flag = false;  // the norm pass reports non-finite grads
    stage_range<DT>(table, n_tensors, ti, f0, f0 + kT8Block, gscale, stage, unused_flag);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = stage[stage_idx(8 * threadIdx.x + j)];
  }
  if (acc != nullptr) {  // read here: up with the state's loads it spilled (GPT-2 shard: 56.5 against 52.5 us)
    float ar[8];
    load_block_f32<true>(acc + k, kBlock8, ar);
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = __fadd_rn(ar[j], g[j]);
  }
  update_block_split<true, SR>(p + k, q.exp_avg + k, q.root + k, q.exp_avg_scale + b, q.root_scale + b,
                               lowp == nullptr ? nullptr : static_cast<unsigned short*>(lowp) + k, lowp_dtype, kBlock8,
                               pr, g, cm, cr, sm, sr, coef, s, key, root_bits, k >> 1);
}

// Any part: the last one, or unaligned state.
template <int DT, int SR>
__device__ __forceinline__ void table8_any(float* p, const zero_state8& q, const float* acc, const zero_tensor* table,
                                           int n_tensors, int64_t shard_start, int64_t k0, int64_t n, float gscale,
                                           void* lowp, int lowp_dtype, float coef, const AdamScalars& s,
                                           uint32_t key, int root_bits, float* stage) {
  const int blen = static_cast<int>(n - k0 < kT8Block ? n - k0 : kT8Block);
  const int64_t f0 = shard_start + k0;
  bool unused_flag = false;
  stage_range<DT>(table, n_tensors, find_tensor_warp(table, n_tensors, f0), f0, f0 + blen, gscale, stage, unused_flag);
  __syncthreads();
  const int q0 = kBlock8 * (threadIdx.x >> 5);
  if (q0 < blen) {
    const int64_t k = k0 + q0, b = k / kBlock8;
    const int left = blen - q0 < kBlock8 ? blen - q0 : kBlock8;
    float pr[8], g[8];
    load_block_f32<false>(p + k, left, pr);
    const uint2 cm = load_codes<false>(q.exp_avg + k, left), cr = load_codes<false>(q.root + k, left);
    const float sm = q.exp_avg_scale[b], sr = q.root_scale[b];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = elem_of<false>(j);
      g[j] = e < left ? stage[stage_idx(q0 + e)] : 0.0f;
      if (acc != nullptr && e < left) g[j] = __fadd_rn(acc[k + e], g[j]);
    }
    update_block_split<false, SR>(p + k, q.exp_avg + k, q.root + k, q.exp_avg_scale + b, q.root_scale + b,
                                  lowp == nullptr ? nullptr : static_cast<unsigned short*>(lowp) + k, lowp_dtype, left,
                                  pr, g, cm, cr, sm, sr, coef, s, key, root_bits, k >> 1);
  }
}

template <int DT, int SR>
__global__ void __launch_bounds__(256, 5)
    adamw_table8_kernel(float* __restrict__ p, zero_state8 q, const float* __restrict__ acc,
                        const zero_tensor* __restrict__ table, int n_tensors, int64_t shard_start, int64_t n,
                        float gscale, const float* __restrict__ dscale, void* __restrict__ lowp, int lowp_dtype,
                        bool state_vec, AdamScalars hs, const zero_adamw_device_state* __restrict__ ds,
                        RoundingBase rnd, const zero_norm_result* __restrict__ clip) {
  __shared__ float stage[kT8Block + kT8Block / 8];
  AdamScalars s = hs;
  if (ds != nullptr && !step_scalars<true>(hs, ds, s)) return;  // the prepared step is skipped
  if (dscale != nullptr) gscale = *dscale;
  float coef = 1.0f;
  if (clip != nullptr) {
    if (!clip->finite) return;  // non-finite grad norm: the step is skipped
    coef = clip->clip_coef;
  }
  const int64_t k0 = static_cast<int64_t>(blockIdx.x) * kT8Block;
  uint32_t key = 0u;
  if (SR != kNearest) key = rounding_key(rnd, ds, 0u, k0 >> 1);
  const bool full = state_vec && n - k0 >= kT8Block;
  if (!ZS_CHECK(k0 < n && (!full || (aligned(p + k0, 32) && aligned(q.exp_avg + k0, 8) && aligned(q.root + k0, 8) &&
                                     (acc == nullptr || aligned(acc + k0, 32)))),
                70, k0))
    return;
  if (full)
    table8_full<DT, SR>(p, q, acc, table, n_tensors, shard_start, k0, gscale, lowp, lowp_dtype, coef, s, key,
                        rnd.root_bits, stage);
  else
    table8_any<DT, SR>(p, q, acc, table, n_tensors, shard_start, k0, n, gscale, lowp, lowp_dtype, coef, s, key,
                        rnd.root_bits, stage);
}

template <int DT, int SR>
static zero_status launch_table8_t(const Table8Args& a, const AdamScalars& s, cudaStream_t st) {
  const bool sv = aligned(a.p, 32) && aligned(a.q.exp_avg, 8) && aligned(a.q.root, 8) &&
                  (a.acc == nullptr || aligned(a.acc, 32));
  adamw_table8_kernel<DT, SR><<<one_pass_blocks(a.n, kT8Block), 256, 0, st>>>(
      a.p, a.q, a.acc, a.table, a.n_tensors, a.shard_start, a.n, a.gscale, a.dscale, a.lowp, a.lowp_dtype, sv, s, a.ds,
      a.rounding, a.clip);
  return check_launch("adamw_table8_kernel");
}

template <int DT>
static zero_status launch_table8_dt(const Table8Args& a, const AdamScalars& s, cudaStream_t st) {
  if (a.rounding.how == kNearest) return launch_table8_t<DT, kNearest>(a, s, st);
  if (a.rounding.how == kRoot7) return launch_table8_t<DT, kRoot7>(a, s, st);
  if (a.rounding.how == kRoot16) return launch_table8_t<DT, kRoot16>(a, s, st);
  return launch_table8_t<DT, kByBeta>(a, s, st);
}

ZS_DEBUG_UNIT(adamw_table8)

zero_status launch_adamw_table8(const Table8Args& a, const AdamScalars& s, cudaStream_t st) {
  if (a.grad_dtype == ZERO_F32) return launch_table8_dt<ZERO_F32>(a, s, st);
  if (a.grad_dtype == ZERO_BF16) return launch_table8_dt<ZERO_BF16>(a, s, st);
  return launch_table8_dt<ZERO_F16>(a, s, st);
}

}  // namespace zs
