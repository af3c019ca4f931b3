// adamw_list.cu -- AdamW over many separate tensors in one launch: each has
// its own fp32 master, moments (fp32, or 8 bits: state8.cuh), grad and
// low-precision copy, and belongs to a parameter group.
//
// Work split: the tensors are cut into chunks of 2048 elements, none across
// two tensors; one block per chunk, a warp per 256 elements (in 8 bits, one
// scale).  A chunk map in device memory, built once with the list, names each
// block's tensor: one dependent read where a search over the list would take
// two or three.
#include "adam.cuh"
#include "common.cuh"
#include "kernels.h"
#include "state8.cuh"
#include "table.cuh"

namespace zs {

// This lane's 8 grads fl(scale * x) of the block whose first element is
// element k of the tensor `src` (NULL: no grad, zeros).
template <int DT>
__device__ __forceinline__ void load_block_grad(const void* src, int64_t k, bool vec, int left, float scale,
                                                float (&g)[8]) {
  constexpr int es = SrcTraits<DT>::esize;
  constexpr int vb = (DT == ZERO_F32) ? 32 : 16;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < 8; ++j) g[j] = 0.0f;
  if (src != nullptr) {
    const char* p = static_cast<const char*>(src) + es * k;
    if (vec && aligned(p, vb)) {
      load8_src<DT>(p + es * 8 * lane, g);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e = elem_of(vec, lane, j);
        if (vec || e < left) g[j] = load_elem<DT>(p, e);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) g[j] = __fmul_rn(scale, g[j]);
}

template <int DT, int BITS, bool SR>
__global__ void __launch_bounds__(256)
    adamw_list_kernel(const zero_list_tensor* __restrict__ list, int n_tensors,
                      const zero_list_chunk* __restrict__ chunks, int64_t n_chunks,
                      const zero_tensor* __restrict__ grads, float gscale, const float* __restrict__ dscale,
                      int lowp_dtype, const __grid_constant__ ListScalars hs,
                      const zero_adamw_device_state* __restrict__ ds, zero_rounding rnd, int64_t step,
                      const zero_norm_result* __restrict__ clip) {
  float coef = 1.0f;
  if (clip != nullptr) {
    if (!clip->finite) return;  // non-finite grad norm: the step is skipped
    coef = clip->clip_coef;
  }
  if (dscale != nullptr) gscale = *dscale;
  const int warp = threadIdx.x >> 5;
  for (int64_t c = blockIdx.x; c < n_chunks; c += gridDim.x) {
    const zero_list_chunk ch = chunks[c];
    if (!ZS_CHECK(ch.tensor >= 0 && ch.tensor < n_tensors && ch.chunk >= 0, 60, c)) continue;
    const zero_list_tensor t = list[ch.tensor];
    const int64_t k = static_cast<int64_t>(ch.chunk) * kListChunk + kBlock8 * warp;
    if (k >= t.numel) continue;
    const int left = static_cast<int>(t.numel - k < kBlock8 ? t.numel - k : kBlock8);
    AdamScalars s;
    if (ds != nullptr) {
      if (!step_scalars<true>(AdamScalars{}, ds + t.group, s)) return;
    } else {
      s = hs.s[t.group];
    }
    constexpr uintptr_t sa = BITS == 8 ? 8 : 32;
    const bool vec = left == kBlock8 && aligned(t.master, 32) && aligned(t.exp_avg, sa) && aligned(t.exp_avg_sq, sa);
    float p[8], g[8];
    load_block_f32(t.master + k, vec, left, p);
    if (BITS == 32) {
      float m[8], v[8];
      load_block_f32(static_cast<float*>(t.exp_avg) + k, vec, left, m);
      load_block_f32(static_cast<float*>(t.exp_avg_sq) + k, vec, left, v);
      load_block_grad<DT>(grads[ch.tensor].ptr, k, vec, left, gscale, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) adam_update(p[j], m[j], v[j], g[j], coef, s);
      store_block_f32(t.master + k, vec, left, p);
      store_block_f32(static_cast<float*>(t.exp_avg) + k, vec, left, m);
      store_block_f32(static_cast<float*>(t.exp_avg_sq) + k, vec, left, v);
    } else {
      uint8_t* cm = static_cast<uint8_t*>(t.exp_avg) + k;
      uint8_t* cr = static_cast<uint8_t*>(t.exp_avg_sq) + k;
      const int64_t b = k / kBlock8;
      uint32_t wm[2], wr[2];
      load_codes(cm, vec, left, wm);
      load_codes(cr, vec, left, wr);
      float sm = t.exp_avg_scale[b], sr = t.root_scale[b];
      load_block_grad<DT>(grads[ch.tensor].ptr, k, vec, left, gscale, g);
      float m[8], r[8];
      decode8(wm, sm, m);
      decode8(wr, sr, r);
      const float inv = __frcp_rn(s.bc2_sqrt);
#pragma unroll
      for (int j = 0; j < 8; ++j) adam_update8(p[j], m[j], r[j], g[j], coef, s, inv);
      uint32_t key = 0u;
      if (SR) key = rounding_key(rnd.seed, ds != nullptr ? ds->step : step, static_cast<uint32_t>(rnd.stream + ch.tensor), k >> 1);
      encode_block<SR>(m, r, vec, key, k >> 1, wm, wr, sm, sr);
      store_block_f32(t.master + k, vec, left, p);
      store_codes(cm, vec, left, wm);
      store_codes(cr, vec, left, wr);
      if ((threadIdx.x & 31) == 0) {
        t.exp_avg_scale[b] = sm;
        t.root_scale[b] = sr;
      }
    }
    if (t.lowp != nullptr) store_block_lowp(static_cast<unsigned short*>(t.lowp) + k, lowp_dtype, vec, left, p);
  }
}

template <int DT, int BITS, bool SR>
static zero_status launch_list_t(const ListArgs& a, const ListScalars& hs, cudaStream_t st) {
  adamw_list_kernel<DT, BITS, SR><<<one_pass_blocks(a.n_chunks, 1), 256, 0, st>>>(
      a.list, a.n_tensors, a.chunks, a.n_chunks, a.grads, a.gscale, a.dscale, a.lowp_dtype, hs, a.ds, a.rounding, a.step,
      a.clip);
  return check_launch("adamw_list_kernel");
}

template <int DT>
static zero_status launch_list_dt(const ListArgs& a, const ListScalars& hs, cudaStream_t st) {
  if (a.state_bits == 32) return launch_list_t<DT, 32, false>(a, hs, st);
  return a.stochastic ? launch_list_t<DT, 8, true>(a, hs, st) : launch_list_t<DT, 8, false>(a, hs, st);
}

ZS_DEBUG_UNIT(adamw_list)

zero_status launch_adamw_list(const ListArgs& a, const ListScalars& hs, cudaStream_t st) {
  if (a.grad_dtype == ZERO_F32) return launch_list_dt<ZERO_F32>(a, hs, st);
  if (a.grad_dtype == ZERO_BF16) return launch_list_dt<ZERO_BF16>(a, hs, st);
  return launch_list_dt<ZERO_F16>(a, hs, st);
}

}  // namespace zs
