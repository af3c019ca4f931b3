// grad_list.cuh -- what the norms of a grads list and its clipping share:
// the chunks of a list and the vectors of a chunk.  Internal.
#pragma once

#include "kernels.h"
#include "list.cuh"
#include "reduce.cuh"

namespace zs {

// The parts of a plan (zero_grad_plan).
struct GradPlan {
  const int32_t* first;        // [n + 1] first wide chunks, their count
  const int32_t* group_first;  // [n_groups + 1] starts in members
  const int32_t* members;      // [n]
  const int32_t* narrow_of;    // [n] a tensor's number in `narrow`, or -1
  const int32_t* narrow;       // [n_narrow] tensors
  int n_wide, n_narrow, chunk;
};
inline GradPlan plan_parts(const GradListArgs& a) {
  GradPlan p;
  p.first = a.plan;
  p.group_first = p.first + a.n + 1;
  p.members = p.group_first + a.n_groups + 1;
  p.narrow_of = p.members + a.n;
  p.narrow = p.narrow_of + a.n;
  p.n_wide = a.n_wide;
  p.n_narrow = a.n_narrow;
  p.chunk = a.chunk;
  return p;
}
inline unsigned grad_blocks(const GradPlan& p, int threads) {
  return static_cast<unsigned>(p.n_wide + (p.n_narrow + threads / 32 - 1) / (threads / 32));
}

// The work of a grid of grad_blocks() blocks of T threads: block b < n_wide has the wide chunk b,
// `chunk` elements of a tensor; each warp of the blocks behind has a narrow
// tensor of its own, so that a list of thousands of small tensors does not
// cost a block's start and end for each.  len == 0: nothing left.
struct GradPiece {
  int tensor, len;
  int64_t k;
  int at;  // its partial
};
__device__ __forceinline__ GradPiece wide_piece(const zero_grad_entry* __restrict__ entries, int n, const GradPlan& p,
                                                int block) {
  GradPiece r;
  r.at = block;
  r.tensor = block_tensor(p.first, n, block);
  r.k = static_cast<int64_t>(block - __ldg(p.first + r.tensor)) * p.chunk;
  const int64_t left = entries[r.tensor].numel - r.k;
  r.len = static_cast<int>(left < p.chunk ? left : p.chunk);
  return r;
}
template <int T>
__device__ __forceinline__ GradPiece narrow_piece(const zero_grad_entry* __restrict__ entries, const GradPlan& p,
                                                  int block) {
  const int j = (block - p.n_wide) * (T / 32) + static_cast<int>(threadIdx.x >> 5);
  if (j >= p.n_narrow) return GradPiece{0, 0, 0, 0};
  const int i = __ldg(p.narrow + j);
  return GradPiece{i, static_cast<int>(entries[i].numel), 0, p.n_wide + j};
}

// A run of `len` elements of ES bytes at p: `head` elements up to the first
// address on the grid of 8 elements' bytes, `vecs` vectors of 8, the tail.
struct Run {
  int head, vecs;
};
template <int ES>
__device__ __forceinline__ Run vector_run(const void* p, int len) {
  constexpr int vb = 8 * ES;
  int h = static_cast<int>(((vb - reinterpret_cast<uintptr_t>(p) % vb) % vb) / ES);
  if (h > len) h = len;
  return Run{h, (len - h) / 8};
}

// The index of thread t's element of the head (threads 0..7) or the tail
// (threads 8..15) of a run, -1 for none.
__device__ __forceinline__ int ragged_element(const Run& r, int len, int t) {
  if (t < 8) return t < r.head ? t : -1;
  const int e = r.head + 8 * r.vecs + t - 8;
  return t < 16 && e < len ? e : -1;
}

// Programmatic dependent launch: a kernel launched by launch_after starts
// while the one before it on the stream still runs, and sees what that one
// wrote after wait_before().  Launched otherwise both do nothing.
__device__ __forceinline__ void wait_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// What an earlier kernel of the stream wrote is read by these alone: as
// volatile assembly they stay behind wait_before() and barriers, which loads
// through the read-only path (__ldg, const __restrict__) and __ldcg need not.
// Of the plan and the entries, which no kernel writes, those are used.
__device__ __forceinline__ uint4 ld16_behind(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}
__device__ __forceinline__ void ld8_behind(const float* p, float (&r)[8]) {
  asm volatile("ld.global.L1::no_allocate.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ double ld_behind(const double* p) {
  double r;
  asm volatile("ld.global.cg.f64 %0, [%1];" : "=d"(r) : "l"(p) : "memory");
  return r;
}
// The bits of one element of a grad.
template <int DT>
__device__ __forceinline__ uint32_t bits_behind(const void* p, int e) {
  if (DT == ZERO_F32) return static_cast<const volatile uint32_t*>(p)[e];
  return static_cast<const volatile unsigned short*>(p)[e];
}
template <int DT>
__device__ __forceinline__ float elem_behind(const void* p, int e) {
  return DT == ZERO_F32 ? __uint_as_float(bits_behind<DT>(p, e)) : half_bits_to_f32<DT>(bits_behind<DT>(p, e));
}

// cluster: the blocks of a thread-block cluster.
template <class... Formal, class... Actual>
inline zero_status launch_after(const char* what, void (*kernel)(Formal...), unsigned blocks, unsigned threads,
                                unsigned cluster, cudaStream_t st, Actual... args) {
  cudaLaunchAttribute attr[2]{};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {cluster, 1, 1};
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<Formal>(args)...);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(ZERO_ECUDA, "%s: %s", what, cudaGetErrorString(e));
  }
  return ZERO_OK;
}

}  // namespace zs
