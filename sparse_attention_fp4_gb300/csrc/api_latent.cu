// C ABI of the latent-attention entry points: argument validation, then kernel launches on
// the caller's stream.
#include <cmath>

#include "latent.cuh"

namespace {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }
inline int from_cuda(cudaError_t e) { return e == cudaSuccess ? FP4IDX_OK : FP4IDX_ERR_CUDA; }

constexpr int64_t kMaxPages = INT32_MAX / fp4idx::kPage;  // slots are int32

int check_attn(const uint16_t* q, int64_t n_rows, int32_t n_heads, int32_t width, const uint16_t* cache,
               int64_t num_pages, const int32_t* page_table, int64_t num_seqs, int32_t max_pages,
               const int32_t* row_seq, float scale, const void* workspace, size_t workspace_bytes,
               const uint16_t* out, const float* lse, const int32_t* status) {
  if (n_rows < 0 || n_heads < 1 || num_pages < 0 || num_seqs < 0 || max_pages < 0) return FP4IDX_ERR_INVALID_ARG;
  if (!std::isfinite(scale)) return FP4IDX_ERR_INVALID_ARG;
  if (width != 512 && width != 576) return FP4IDX_ERR_UNSUPPORTED;
  if (n_heads > FP4IDX_LATENT_MAX_HEADS || n_rows > FP4IDX_LATENT_MAX_ROWS) return FP4IDX_ERR_UNSUPPORTED;
  if (num_pages > kMaxPages || max_pages > kMaxPages || num_seqs > INT32_MAX) return FP4IDX_ERR_UNSUPPORTED;
  if (n_rows == 0) return FP4IDX_OK;  // (a step without a sequence has no table either)
  if (num_pages < 1 || num_seqs < 1 || max_pages < 1) return FP4IDX_ERR_INVALID_ARG;
  if (!q || !cache || !page_table || !row_seq || !out || !workspace) return FP4IDX_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(cache) || !aligned16(out) || !aligned16(workspace)) return FP4IDX_ERR_INVALID_ARG;
  if (!aligned4(page_table) || !aligned4(row_seq) || !aligned4(lse) || !aligned4(status))
    return FP4IDX_ERR_INVALID_ARG;
  if (workspace_bytes < fp4idx::latent_attn_workspace_bytes(n_rows, n_heads)) return FP4IDX_ERR_WORKSPACE;
  return FP4IDX_OK;
}

}  // namespace

extern "C" {

int fp4idx_plan_step(const int32_t* cached_lens, const int32_t* new_lens, int64_t n_seqs, int32_t ratio,
                     const int32_t* free_pages, int64_t n_free, const int32_t* free_head, int32_t* page_table,
                     int32_t max_pages, int32_t* q_positions, int32_t* row_seq, int32_t* context_lens,
                     int64_t max_rows, int32_t* store_positions, int32_t* store_slots, int64_t max_stores,
                     int32_t* cu_rows, int32_t* cu_context, int32_t* counts, int32_t* status_dev, void* stream) {
  if (n_seqs < 0 || n_free < 0 || max_pages < 1 || max_rows < 0 || max_stores < 0 || ratio < 1 || ratio > 64)
    return FP4IDX_ERR_INVALID_ARG;
  if (n_seqs > 65536 || max_pages > kMaxPages || n_free > INT32_MAX || max_rows > (1 << 30) || max_stores > (1 << 30))
    return FP4IDX_ERR_UNSUPPORTED;
  if (!cu_rows || !cu_context || !counts) return FP4IDX_ERR_INVALID_ARG;
  if (n_seqs > 0 && (!cached_lens || !new_lens || !page_table)) return FP4IDX_ERR_INVALID_ARG;
  if (n_free > 0 && !free_pages) return FP4IDX_ERR_INVALID_ARG;
  if (max_rows > 0 && (!q_positions || !row_seq || !context_lens)) return FP4IDX_ERR_INVALID_ARG;
  if (max_stores > 0 && (!store_positions || !store_slots)) return FP4IDX_ERR_INVALID_ARG;
  const void* ptrs[] = {cached_lens, new_lens,        free_pages,  free_head, page_table, q_positions, row_seq,
                        context_lens, store_positions, store_slots, cu_rows,   cu_context, counts,      status_dev};
  for (const void* p : ptrs)
    if (!aligned4(p)) return FP4IDX_ERR_INVALID_ARG;
  fp4idx::PlanArgs a{cached_lens, new_lens, free_pages, free_head, page_table, q_positions, row_seq, context_lens,
                     store_positions, store_slots, cu_rows, cu_context, counts, status_dev, (int32_t)n_seqs, ratio,
                     (int32_t)n_free, max_pages, (int32_t)max_rows, (int32_t)max_stores};
  return from_cuda(fp4idx::launch_plan_step(a, as_stream(stream)));
}

int fp4idx_store_latent(const uint16_t* kv, int64_t n_rows, int32_t width, const int32_t* positions,
                        const int32_t* slots, const uint16_t* norm_w, float eps, const uint16_t* cos_sin,
                        int32_t max_pos, uint16_t* cache, int64_t num_pages, int32_t* status_dev, void* stream) {
  if (n_rows < 0 || num_pages < 0 || max_pos <= 0) return FP4IDX_ERR_INVALID_ARG;
  if (width != 512 && width != 576) return FP4IDX_ERR_UNSUPPORTED;
  if (num_pages > kMaxPages) return FP4IDX_ERR_UNSUPPORTED;
  if (n_rows == 0) return FP4IDX_OK;
  if (!kv || !positions || !slots || !norm_w || !cos_sin || !cache) return FP4IDX_ERR_INVALID_ARG;
  if (!aligned16(kv) || !aligned16(norm_w) || !aligned16(cos_sin) || !aligned16(cache) || !aligned4(positions) ||
      !aligned4(slots) || !aligned4(status_dev))
    return FP4IDX_ERR_INVALID_ARG;
  return from_cuda(fp4idx::launch_store_latent(kv, n_rows, width, positions, slots, norm_w, eps, cos_sin, max_pos,
                                               cache, num_pages, status_dev, as_stream(stream)));
}

size_t fp4idx_latent_attn_workspace_bytes(int64_t max_rows, int32_t n_heads) {
  if (max_rows < 0 || max_rows > FP4IDX_LATENT_MAX_ROWS || n_heads < 1 || n_heads > FP4IDX_LATENT_MAX_HEADS) return 0;
  return fp4idx::latent_attn_workspace_bytes(max_rows, n_heads);
}

int fp4idx_latent_attn_topk(const uint16_t* q, int64_t n_rows, int32_t n_heads, int32_t width, const uint16_t* cache,
                            int64_t num_pages, const int32_t* page_table, int64_t num_seqs, int32_t max_pages,
                            const int32_t* row_seq, const int32_t* topk_idx, int32_t k, const int32_t* context_lens,
                            float scale, void* workspace, size_t workspace_bytes, uint16_t* out, float* lse,
                            int32_t* status_dev, void* stream) {
  if (k < 1 || k > FP4IDX_MAX_TOPK) return FP4IDX_ERR_INVALID_ARG;
  int st = check_attn(q, n_rows, n_heads, width, cache, num_pages, page_table, num_seqs, max_pages, row_seq, scale,
                      workspace, workspace_bytes, out, lse, status_dev);
  if (st != FP4IDX_OK || n_rows == 0) return st;
  if (!topk_idx || !aligned4(topk_idx) || !aligned4(context_lens)) return FP4IDX_ERR_INVALID_ARG;
  fp4idx::LatentArgs a{};
  a.q = q; a.cache = cache; a.page_table = page_table; a.row_seq = row_seq; a.idx = topk_idx;
  a.context_lens = context_lens; a.out = out; a.lse = lse; a.status = status_dev; a.workspace = workspace;
  a.num_pages = (int32_t)num_pages; a.num_seqs = (int32_t)num_seqs; a.max_pages = max_pages; a.n_rows = (int32_t)n_rows;
  a.heads = n_heads; a.k = k; a.scale = scale;
  return from_cuda(fp4idx::launch_latent_attn(a, width, true, as_stream(stream)));
}

int fp4idx_latent_attn(const uint16_t* q, int64_t n_rows, int32_t n_heads, int32_t width, const uint16_t* cache,
                       int64_t num_pages, const int32_t* page_table, int64_t num_seqs, int32_t max_pages,
                       const int32_t* row_seq, const int32_t* context_lens, int32_t max_context,
                       const uint32_t* tree_mask, int32_t mask_words, float scale, void* workspace,
                       size_t workspace_bytes, uint16_t* out, float* lse, int32_t* status_dev, void* stream) {
  if (max_context < 0 || mask_words < 0) return FP4IDX_ERR_INVALID_ARG;
  if ((tree_mask == nullptr) != (mask_words == 0)) return FP4IDX_ERR_INVALID_ARG;
  if (mask_words > FP4IDX_LATENT_MAX_TREE_WORDS) return FP4IDX_ERR_UNSUPPORTED;
  int st = check_attn(q, n_rows, n_heads, width, cache, num_pages, page_table, num_seqs, max_pages, row_seq, scale,
                      workspace, workspace_bytes, out, lse, status_dev);
  if (st != FP4IDX_OK) return st;
  if ((int64_t)max_context > (int64_t)max_pages * fp4idx::kPage) return FP4IDX_ERR_INVALID_ARG;
  if (n_rows == 0) return FP4IDX_OK;
  if (!context_lens || !aligned4(context_lens) || !aligned4(tree_mask)) return FP4IDX_ERR_INVALID_ARG;
  fp4idx::LatentArgs a{};
  a.q = q; a.cache = cache; a.page_table = page_table; a.row_seq = row_seq; a.context_lens = context_lens;
  a.tree = tree_mask; a.words = mask_words; a.max_context = max_context; a.out = out; a.lse = lse;
  a.status = status_dev; a.workspace = workspace; a.num_pages = (int32_t)num_pages; a.num_seqs = (int32_t)num_seqs;
  a.max_pages = max_pages; a.n_rows = (int32_t)n_rows; a.heads = n_heads; a.scale = scale;
  return from_cuda(fp4idx::launch_latent_attn(a, width, false, as_stream(stream)));
}

int fp4idx_latent_prefill(const uint16_t* q, int64_t n_q, int32_t n_heads, const uint16_t* kv, int64_t n_kv,
                          const uint16_t* k_rope, const int32_t* cu_q, const int32_t* cu_kv, int64_t n_seqs,
                          int32_t max_q, int32_t max_kv, float scale, uint16_t* out, float* lse, int32_t* status_dev,
                          void* stream) {
  if (n_q < 0 || n_kv < 0 || n_seqs < 0 || max_q < 0 || max_kv < 0 || n_heads < 1 || !std::isfinite(scale))
    return FP4IDX_ERR_INVALID_ARG;
  if (n_heads > 1024 || n_seqs > 65535 || n_q > (1 << 24) || n_kv > (1 << 24)) return FP4IDX_ERR_UNSUPPORTED;
  if (n_q == 0 || n_seqs == 0 || max_q == 0) return FP4IDX_OK;
  if (!q || !cu_q || !cu_kv || !out) return FP4IDX_ERR_INVALID_ARG;
  if (n_kv > 0 && (!kv || !k_rope)) return FP4IDX_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(kv) || !aligned16(k_rope) || !aligned16(out) || !aligned4(cu_q) ||
      !aligned4(cu_kv) || !aligned4(lse) || !aligned4(status_dev))
    return FP4IDX_ERR_INVALID_ARG;
  fp4idx::PrefillArgs a{};
  a.q = q; a.kv = kv; a.k_rope = k_rope; a.cu_q = cu_q; a.cu_kv = cu_kv; a.out = out; a.lse = lse;
  a.status = status_dev; a.n_q = (int32_t)n_q; a.n_kv = (int32_t)n_kv; a.n_seqs = (int32_t)n_seqs; a.heads = n_heads;
  a.max_q = max_q < a.n_q ? max_q : a.n_q; a.max_kv = max_kv; a.scale = scale;  // (loose bounds launch no more)
  return from_cuda(fp4idx::launch_latent_prefill(a, as_stream(stream)));
}

}  // extern "C"
