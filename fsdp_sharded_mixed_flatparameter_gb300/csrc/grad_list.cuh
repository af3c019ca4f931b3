// grad_list.cuh -- what the norms of a grads list and its clipping share:
// the chunks of a list and the vectors of a chunk.  Internal.
#pragma once

#include "list.cuh"
#include "reduce.cuh"

namespace zs {

constexpr int kGradThreads = 256;

// The parts of a plan (zero_grad_plan).
struct GradPlan {
  const int32_t* first;        // [n + 1] first chunks, their count
  const int32_t* group_first;  // [n_groups + 1] starts in members
  const int32_t* members;      // [n]
};
__host__ __device__ inline GradPlan plan_parts(const int32_t* plan, int n, int n_groups) {
  return GradPlan{plan, plan + n + 1, plan + n + 1 + n_groups + 1};
}

// A chunk: elements [k, k + len) of a tensor.
struct GradChunk {
  int tensor;
  int64_t k;
  int len;
};
__device__ __forceinline__ GradChunk grad_chunk(const zero_grad_entry* __restrict__ entries,
                                                const int32_t* __restrict__ first, int n, int chunk, int c) {
  GradChunk r;
  r.tensor = block_tensor(first, n, c);
  r.k = static_cast<int64_t>(c - __ldg(first + r.tensor)) * chunk;
  const int64_t left = entries[r.tensor].numel - r.k;
  r.len = static_cast<int>(left < chunk ? left : chunk);
  return r;
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

// The index of this thread's element of the head (threads 0..7) or the tail
// (threads 8..15) of a run, -1 for none.
__device__ __forceinline__ int ragged_element(const Run& r, int len) {
  const int t = threadIdx.x;
  if (t < 8) return t < r.head ? t : -1;
  const int e = r.head + 8 * r.vecs + t - 8;
  return t < 16 && e < len ? e : -1;
}

}  // namespace zs
