// Host launchers of the step plan, the latent cache and latent attention, called by their C
// ABI (api_latent.cu).
#pragma once

#include "launchers.cuh"

namespace fp4idx {

// How many clusters of `size` CTAs of `threads` threads and `smem` bytes of dynamic shared
// memory fit on the current device at once (none of a size that it cannot place), computed once
// per (kernel, size, device).
cudaError_t resident_clusters(const void* kernel, int size, int threads, size_t smem, int* out);

// A launch, of clusters of `cluster` CTAs along x, that may begin while the one before it on the stream ends: the kernel waits
// (griddepcontrol.wait) before its first access to global memory, and reads none of it as
// read-only data, which the compiler may move above the wait.
template <class... A, class... B>
cudaError_t launch_early(void (*kernel)(A...), dim3 grid, int threads, size_t smem, int cluster, cudaStream_t stream,
                         const B&... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<A>(args)...);
}

struct PlanArgs {
  const int32_t *cached, *fresh, *free_pages, *free_head;
  int32_t *page_table, *q_positions, *row_seq, *context_lens, *store_positions, *store_slots, *cu_rows, *cu_context;
  int32_t *counts, *status;
  int32_t n_seqs, ratio, n_free, max_pages, max_rows, max_stores;
};
cudaError_t launch_plan_step(const PlanArgs& a, cudaStream_t stream);
cudaError_t launch_store_latent(const uint16_t* kv, int64_t n_rows, int32_t width, const int32_t* positions,
                                const int32_t* slots, const uint16_t* norm_w, float eps, const uint16_t* cos_sin,
                                int32_t max_pos, uint16_t* cache, int64_t num_pages, int32_t* status,
                                cudaStream_t stream);
struct LatentArgs {
  const uint16_t *q, *cache;
  const int32_t *page_table, *row_seq, *context_lens;
  const int32_t* idx;    // selected positions [n_rows, k]; null: the whole context
  const uint32_t* tree;  // drafted tokens' masks [n_rows, words] (nullable)
  uint16_t* out;
  float* lse;
  int32_t* status;
  void* workspace;
  int32_t num_pages, num_seqs, max_pages, n_rows, heads, k, words, max_context;
  float scale;
};
size_t latent_attn_workspace_bytes(int64_t n_rows, int32_t n_heads);
cudaError_t launch_latent_attn(const LatentArgs& a, int32_t width, bool selected, cudaStream_t stream);
struct PrefillArgs {
  const uint16_t *q, *kv, *k_rope;
  const int32_t *cu_q, *cu_kv;
  uint16_t* out;
  float* lse;
  int32_t* status;
  int32_t n_q, n_kv, n_seqs, heads, max_q, max_kv;
  float scale;
};
cudaError_t launch_latent_prefill(const PrefillArgs& a, cudaStream_t stream);

}  // namespace fp4idx
