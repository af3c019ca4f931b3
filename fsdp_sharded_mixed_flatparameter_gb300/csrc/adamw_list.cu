// adamw_list.cu -- AdamW over many separate tensors in one launch: each has
// its own fp32 master and moments, grad and low-precision copy, and belongs to
// a parameter group.  (Moments in 8 bits: adamw_list8.cu.)
//
// Work split: the tensors are cut into chunks of 1024 elements, none across
// two tensors; one block of 128 threads per chunk, a warp per 256 elements, 8
// per lane (32-byte accesses).  The block's tensor is found by a search over
// the tensors' first chunks (list.cuh).
//
// Bound by HBM: 28 bytes an element with 16-bit grads and copy.  Four layers
// of Llama-7B with embedding and head (1.07e9 elements): 4.25 ms = 7.06 TB/s;
// 4000 log-uniform tensors (302e6): 1.20 ms = 7.04 TB/s; GPT-2 small (148
// tensors, 124e6): 0.498 ms = 6.99 TB/s.  Ten blocks per SM (48 registers)
// against eight (64): the ragged list 1.21 against 1.25 ms, large tensors the
// same; chunks of 2048 in blocks of 256: 1.27.  Four layers of fp32 moments
// with grads off the 16-byte grid: 4.27 ms.
#include "adam.cuh"
#include "common.cuh"
#include "kernels.h"
#include "list.cuh"

namespace zs {

template <int DT, bool VEC>
__device__ __forceinline__ void list_block(const zero_list_tensor& t, const void* grad, int64_t k, int64_t rest,
                                           float gscale, float coef, const AdamScalars& s, int lowp_dtype) {
  const int left = static_cast<int>(rest < kBlock8 ? rest : kBlock8);
  float p[8], m[8], v[8], g[8];
  float* const pk = t.master + k;
  float* const mk = static_cast<float*>(t.exp_avg) + k;
  float* const vk = static_cast<float*>(t.exp_avg_sq) + k;
  load_block_f32<VEC>(pk, left, p);
  load_block_f32<VEC>(mk, left, m);
  load_block_f32<VEC>(vk, left, v);
  load_block_grad<DT, VEC>(grad, k, rest, gscale, g);
#pragma unroll
  for (int j = 0; j < 8; ++j) adam_update(p[j], m[j], v[j], g[j], coef, s);
  store_block_f32<VEC>(pk, left, p);
  store_block_f32<VEC>(mk, left, m);
  store_block_f32<VEC>(vk, left, v);
  if (t.lowp != nullptr) store_block_lowp<VEC>(static_cast<unsigned short*>(t.lowp) + k, lowp_dtype, left, p);
}

template <int DT>
__global__ void __launch_bounds__(kListThreads, 10)
    adamw_list_kernel(const zero_list_tensor* __restrict__ list, int n_tensors,
                      const int32_t* __restrict__ first_chunk, const zero_tensor* __restrict__ grads, float gscale,
                      const float* __restrict__ dscale, int lowp_dtype, const __grid_constant__ ListScalars hs,
                      const zero_adamw_device_state* __restrict__ ds, const zero_norm_result* __restrict__ clip) {
  const int tensor = block_tensor(first_chunk, n_tensors, blockIdx.x);
  const int chunk = blockIdx.x - __ldg(first_chunk + tensor);
  const zero_list_tensor t = list[tensor];
  const void* grad = grads[tensor].ptr;
  if (!ZS_CHECK(chunk >= 0 && chunk < (t.numel + kListChunk - 1) / kListChunk, 60, blockIdx.x)) return;
  float coef = 1.0f;
  if (clip != nullptr) {
    if (!clip->finite) return;  // non-finite grad norm: the step is skipped
    coef = clip->clip_coef;
  }
  if (dscale != nullptr) gscale = *dscale;
  const int64_t k = static_cast<int64_t>(chunk) * kListChunk + kBlock8 * (threadIdx.x >> 5);
  const int64_t left = t.numel - k;
  if (left <= 0) return;
  AdamScalars s;
  if (!group_scalars(hs, ds, t.group, s)) return;
  if (left >= kBlock8 && aligned(t.master, 32) && aligned(t.exp_avg, 32) && aligned(t.exp_avg_sq, 32))
    list_block<DT, true>(t, grad, k, left, gscale, coef, s, lowp_dtype);
  else
    list_block<DT, false>(t, grad, k, left, gscale, coef, s, lowp_dtype);
}

template <int DT>
static zero_status launch_list_t(const ListArgs& a, const ListScalars& hs, cudaStream_t st) {
  adamw_list_kernel<DT><<<static_cast<unsigned>(a.n_chunks), kListThreads, 0, st>>>(
      a.list, a.n_tensors, a.first_chunk, a.grads, a.gscale, a.dscale, a.lowp_dtype, hs, a.ds, a.clip);
  return check_launch("adamw_list_kernel");
}

ZS_DEBUG_UNIT(adamw_list)

zero_status launch_adamw_list(const ListArgs& a, const ListScalars& hs, cudaStream_t st) {
  if (a.state_bits == 8) return launch_adamw_list8(a, hs, st);
  if (a.grad_dtype == ZERO_F32) return launch_list_t<ZERO_F32>(a, hs, st);
  if (a.grad_dtype == ZERO_BF16) return launch_list_t<ZERO_BF16>(a, hs, st);
  return launch_list_t<ZERO_F16>(a, hs, st);
}

}  // namespace zs
