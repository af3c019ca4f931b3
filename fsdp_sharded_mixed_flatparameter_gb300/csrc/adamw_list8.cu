// adamw_list8.cu -- AdamW over many separate tensors in one launch, with the
// moments in 8 bits (state8.cuh).  The work split is adamw_list.cu's: a block
// per chunk of 1024 elements, a warp per 256, which here is one scale: its
// maximum is one warp reduction, nothing is shared between warps.
//
// 16 bytes an element with 16-bit grads and copy, and 52 instructions (65
// with stochastic rounding, 68 with 16 bits for the root): near the
// bandwidth's and the issue rate's limit at once.  Eight layers of Llama-7B
// (1.88e9 elements), stochastic: 4.50 ms = 6.72 TB/s (16 bits: 4.55; with the
// bits chosen in the kernel by the device's betas 4.60, 4.71 with 16 for the
// root, 4.86 with 16 for both); four
// layers (1.07e9): 2.49 ms to nearest (6.93 TB/s), 2.58 stochastic, 2.51 to
// nearest with grads off the 16-byte grid; fp32 grads 2.71 on and off theirs.
// 4000 log-uniform tensors (302e6): 0.81 ms = 5.98 TB/s, where short last
// chunks leave warps idle and the search takes a second round; GPT-2 small,
// stochastic: 0.317 ms = 6.32 TB/s.
//
// The way there, 1.88e9 elements, stochastic: 9.62 ms at 100 registers (one
// code for full and short blocks); 6.09 with the two apart at 64 registers;
// 5.62 with paired arithmetic and the hardware root and reciprocal (43
// instructions to nearest, 74 before); 4.84 at five blocks of 256 per SM (48
// registers) instead of four; 4.76 with the search in place of a chunk map;
// 4.69 with blocks of 128; 4.66 with the rounding key hashed on the host; 4.57
// with the stochastic codes collected by byte permutation; 4.51 with one
// search per block; 4.41 with its last round over 128 candidates; 4.45 with the
// root taken to the correctly rounded one by a Newton step in place of the
// hardware's (by the compiler's sequence: 4.55), so that the stored codes are
// those of the formula and not of the hardware's last bit; 4.50 with the blocks of
// small roots computed larger (kLift).  Not kept:
// asynchronous copies into shared memory, a block's chunks in a pipeline of two
// or three stages (6.2 to 6.9 ms at the first arithmetic, against 6.1: their
// addressing and waits are instructions).
#include "common.cuh"
#include "kernels.h"
#include "list.cuh"

namespace zs {

template <int DT, int SR, bool VEC>
__device__ __forceinline__ void list8_block(const zero_list_tensor& t, const void* grad, int64_t k, int64_t rest,
                                            float gscale, float coef, const AdamScalars& s, int lowp_dtype,
                                            uint32_t key, int root_bits) {
  const int left = static_cast<int>(rest < kBlock8 ? rest : kBlock8);
  float p[8], g[8];
  float* const pk = t.master + k;
  uint8_t* const qm = static_cast<uint8_t*>(t.exp_avg) + k;
  uint8_t* const qr = static_cast<uint8_t*>(t.exp_avg_sq) + k;
  float* const ms = t.exp_avg_scale + k / kBlock8;
  float* const rs = t.root_scale + k / kBlock8;
  load_block_f32<VEC>(pk, left, p);
  const uint2 cm = load_codes<VEC>(qm, left), cr = load_codes<VEC>(qr, left);
  const float sm = *ms, sr = *rs;
  load_block_grad<DT, VEC>(grad, k, rest, gscale, g);
  update_block<VEC, SR, kAnyRoots>(pk, qm, qr, ms, rs,
                                   t.lowp == nullptr ? nullptr : static_cast<unsigned short*>(t.lowp) + k, lowp_dtype,
                                   left, p, g, cm, cr, sm, sr, coef, s, key, root_bits, k >> 1);
}

template <int DT, int SR>
__global__ void __launch_bounds__(kListThreads, 10)
    adamw_list8_kernel(const zero_list_tensor* __restrict__ list, int n_tensors,
                       const int32_t* __restrict__ first_chunk, const zero_tensor* __restrict__ grads, float gscale,
                       const float* __restrict__ dscale, int lowp_dtype, const __grid_constant__ ListScalars hs,
                       const zero_adamw_device_state* __restrict__ ds, RoundingBase rnd,
                       const zero_norm_result* __restrict__ clip, int clips) {
  const int tensor = block_tensor(first_chunk, n_tensors, blockIdx.x);
  const int chunk = blockIdx.x - __ldg(first_chunk + tensor);
  const zero_list_tensor t = list[tensor];
  const void* grad = grads[tensor].ptr;
  if (!ZS_CHECK(chunk >= 0 && chunk < (t.numel + kListChunk - 1) / kListChunk, 90, blockIdx.x)) return;
  float coef = 1.0f;
  if (clip != nullptr) {
    if (!clip[clips].finite) return;  // non-finite grad norm: the step is skipped
    coef = clip[clips != 0 ? t.group : 0].clip_coef;
  }
  if (dscale != nullptr) gscale = *dscale;
  const int64_t k = static_cast<int64_t>(chunk) * kListChunk + kBlock8 * (threadIdx.x >> 5);
  const int64_t left = t.numel - k;
  if (left <= 0) return;
  AdamScalars s;
  if (!group_scalars(hs, ds, t.group, s)) return;
  uint32_t key = 0u;
  if (SR != kNearest) key = rounding_key(rnd, ds, tensor, k >> 1);
  if (left >= kBlock8 && aligned(t.master, 32) && aligned(t.exp_avg, 8) && aligned(t.exp_avg_sq, 8))
    list8_block<DT, SR, true>(t, grad, k, left, gscale, coef, s, lowp_dtype, key, rnd.root_bits);
  else
    list8_block<DT, SR, false>(t, grad, k, left, gscale, coef, s, lowp_dtype, key, rnd.root_bits);
}

template <int DT, int SR>
static zero_status launch_list8_t(const ListArgs& a, const ListScalars& hs, cudaStream_t st) {
  adamw_list8_kernel<DT, SR><<<static_cast<unsigned>(a.n_chunks), kListThreads, 0, st>>>(
      a.list, a.n_tensors, a.first_chunk, a.grads, a.gscale, a.dscale, a.lowp_dtype, hs, a.ds, a.rounding, a.clip, a.clips);
  return check_launch("adamw_list8_kernel");
}

ZS_DEBUG_UNIT(adamw_list8)

template <int DT>
static zero_status launch_list8_dt(const ListArgs& a, const ListScalars& hs, cudaStream_t st) {
  if (a.rounding.how == kNearest) return launch_list8_t<DT, kNearest>(a, hs, st);
  if (a.rounding.how == kRoot7) return launch_list8_t<DT, kRoot7>(a, hs, st);
  if (a.rounding.how == kRoot16) return launch_list8_t<DT, kRoot16>(a, hs, st);
  return launch_list8_t<DT, kByBeta>(a, hs, st);
}

zero_status launch_adamw_list8(const ListArgs& a, const ListScalars& hs, cudaStream_t st) {
  if (a.grad_dtype == ZERO_F32) return launch_list8_dt<ZERO_F32>(a, hs, st);
  if (a.grad_dtype == ZERO_BF16) return launch_list8_dt<ZERO_BF16>(a, hs, st);
  return launch_list8_dt<ZERO_F16>(a, hs, st);
}

}  // namespace zs
