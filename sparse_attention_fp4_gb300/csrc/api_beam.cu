// C ABI of the beam selection and of the page pool's operators: argument validation, then kernel
// launches on the caller's stream.
#include "beam.cuh"

namespace {

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }
inline int from_cuda(cudaError_t e) { return e == cudaSuccess ? FP4IDX_OK : FP4IDX_ERR_CUDA; }

// Page tables of fork and compaction.
int check_pool(int64_t num_pages, int32_t max_pages, int32_t ratio, int64_t n_free, const void* free_pages,
               const void* pinned) {
  if (num_pages < 1 || max_pages < 1 || ratio < 1 || ratio > 64 || n_free < 0) return FP4IDX_ERR_INVALID_ARG;
  if (num_pages > FP4IDX_MAX_POOL_PAGES || max_pages > INT32_MAX / fp4idx::kPage || n_free > INT32_MAX)
    return FP4IDX_ERR_UNSUPPORTED;
  if ((n_free > 0 && !free_pages) || !aligned(free_pages, 4) || !aligned(pinned, 4)) return FP4IDX_ERR_INVALID_ARG;
  return FP4IDX_OK;
}

}  // namespace

extern "C" {

size_t fp4idx_beam_select_workspace_bytes(int64_t max_rows, int32_t vocab, int32_t k) {
  if (max_rows < 0 || max_rows > FP4IDX_BEAM_MAX_ROWS || vocab < 1 || vocab > FP4IDX_BEAM_MAX_VOCAB || k < 1 ||
      k > FP4IDX_BEAM_MAX_K)
    return 0;
  return fp4idx::beam_select_workspace_bytes(max_rows, vocab, k);
}

int fp4idx_beam_select(const void* logits, int32_t logits_type, int64_t logits_stride, int32_t vocab,
                       const float* scores, int64_t n_rows, int32_t n_beams, int32_t k, const int32_t* done,
                       int32_t end_token, void* workspace, size_t workspace_bytes, float* out_scores,
                       int32_t* out_rows, int32_t* out_tokens, int32_t* done_out, int32_t* status_dev, void* stream) {
  if (n_rows < 0 || n_beams < 1 || k < 1 || vocab < 1 || logits_stride < vocab || end_token < -1 || end_token >= vocab)
    return FP4IDX_ERR_INVALID_ARG;
  if (logits_type < 0 || logits_type > 2 || n_beams > FP4IDX_BEAM_MAX_BEAMS || k > FP4IDX_BEAM_MAX_K ||
      vocab > FP4IDX_BEAM_MAX_VOCAB || n_rows > FP4IDX_BEAM_MAX_ROWS || logits_stride > ((int64_t)1 << 40))
    return FP4IDX_ERR_UNSUPPORTED;
  if (n_rows % n_beams != 0 || (done && end_token < 0)) return FP4IDX_ERR_INVALID_ARG;
  if (n_rows == 0) return FP4IDX_OK;
  if (!logits || !scores || !out_scores || !out_rows || !out_tokens || !workspace) return FP4IDX_ERR_INVALID_ARG;
  const void* ptrs[] = {scores, done, out_scores, out_rows, out_tokens, done_out, status_dev};
  for (const void* p : ptrs)
    if (!aligned(p, 4)) return FP4IDX_ERR_INVALID_ARG;
  if (!aligned(logits, logits_type == 2 ? 4 : 2) || !aligned(workspace, 16)) return FP4IDX_ERR_INVALID_ARG;
  if (workspace_bytes < fp4idx::beam_select_workspace_bytes(n_rows, vocab, k)) return FP4IDX_ERR_WORKSPACE;
  fp4idx::BeamArgs a{};
  a.logits = logits; a.scores = scores; a.done = done; a.out_scores = out_scores; a.out_rows = out_rows;
  a.out_tokens = out_tokens; a.done_out = done_out; a.status = status_dev; a.stride = logits_stride;
  a.n_rows = (int32_t)n_rows; a.vocab = vocab; a.beams = n_beams; a.k = k; a.end_token = end_token;
  return from_cuda(fp4idx::launch_beam_select(a, logits_type, workspace, as_stream(stream)));
}

int fp4idx_fork_pages(const int32_t* page_table, const int32_t* cached_lens, int64_t n_old, int32_t max_pages,
                      int32_t ratio, const int32_t* parents, int64_t n_new, int64_t num_pages, const uint32_t* pinned,
                      int32_t* free_pages, int64_t n_free, const int32_t* free_head, int32_t* page_table_out,
                      int32_t* cached_out, int32_t* copy_src, int32_t* copy_dst, int32_t* counts, int32_t* status_dev,
                      void* stream) {
  if (n_old < 0 || n_new < 0) return FP4IDX_ERR_INVALID_ARG;
  const int st = check_pool(num_pages, max_pages, ratio, n_free, free_pages, pinned);
  if (st != FP4IDX_OK) return st;
  if (n_old > FP4IDX_FORK_MAX_ROWS || n_new > FP4IDX_FORK_MAX_ROWS) return FP4IDX_ERR_UNSUPPORTED;
  if (!counts || (n_old > 0 && (!page_table || !cached_lens))) return FP4IDX_ERR_INVALID_ARG;
  if (n_new > 0 && (!parents || !page_table_out || !cached_out || !copy_src || !copy_dst)) return FP4IDX_ERR_INVALID_ARG;
  if (n_old > 0 && n_new > 0 && (page_table == page_table_out || cached_lens == cached_out)) return FP4IDX_ERR_INVALID_ARG;
  const void* ptrs[] = {page_table, cached_lens, parents,  free_head, page_table_out,
                        cached_out, copy_src,    copy_dst, counts,    status_dev};
  for (const void* p : ptrs)
    if (!aligned(p, 4)) return FP4IDX_ERR_INVALID_ARG;
  fp4idx::ForkArgs a{page_table, cached_lens, parents, pinned, free_pages, free_head, page_table_out, cached_out,
                     copy_src, copy_dst, counts, status_dev, (int32_t)n_old, (int32_t)n_new, max_pages, ratio,
                     (int32_t)num_pages, (int32_t)n_free};
  return from_cuda(fp4idx::launch_fork_pages(a, as_stream(stream)));
}

int fp4idx_copy_pages(const int32_t* src, const int32_t* dst, int64_t n_copies, const int32_t* count,
                      void* const* regions, const int64_t* page_bytes, int32_t n_regions, int64_t num_pages,
                      int32_t* status_dev, void* stream) {
  if (n_copies < 0 || n_regions < 0 || num_pages < 0) return FP4IDX_ERR_INVALID_ARG;
  if (n_copies > (1 << 24) || n_regions > FP4IDX_COPY_MAX_REGIONS || num_pages > INT32_MAX) return FP4IDX_ERR_UNSUPPORTED;
  if (n_regions > 0 && (!regions || !page_bytes)) return FP4IDX_ERR_INVALID_ARG;
  if (n_copies > 0 && (!src || !dst)) return FP4IDX_ERR_INVALID_ARG;
  if (!aligned(src, 4) || !aligned(dst, 4) || !aligned(count, 4) || !aligned(status_dev, 4)) return FP4IDX_ERR_INVALID_ARG;
  fp4idx::Regions r{};
  for (int32_t c = 0; c < n_regions; c++) {
    if ((!regions[c] && num_pages > 0) || !aligned(regions[c], 16) || page_bytes[c] < 16 || page_bytes[c] % 16 != 0)
      return FP4IDX_ERR_INVALID_ARG;
    if (page_bytes[c] > (1 << 30)) return FP4IDX_ERR_UNSUPPORTED;
    r.base[c] = static_cast<uint8_t*>(regions[c]);
    r.vecs[c] = (int32_t)(page_bytes[c] / 16);
  }
  r.n = n_regions;
  if (n_copies == 0 || n_regions == 0 || num_pages == 0) return FP4IDX_OK;
  return from_cuda(fp4idx::launch_move_pages(src, dst, n_copies, count, r, num_pages, status_dev, as_stream(stream)));
}

size_t fp4idx_compact_pages_workspace_bytes(int64_t num_pages) {
  if (num_pages < 1 || num_pages > FP4IDX_MAX_POOL_PAGES) return 0;
  return (size_t)num_pages * sizeof(int32_t);
}

int fp4idx_compact_pages(const int32_t* page_table, const int32_t* cached_lens, int64_t n_seqs, int32_t max_pages,
                         int32_t ratio, int64_t num_pages, const uint32_t* pinned, void* workspace,
                         size_t workspace_bytes, int32_t* free_pages, int64_t n_free, int32_t* page_table_out,
                         int32_t* move_src, int32_t* move_dst, int64_t max_moves, int32_t* counts, int32_t* status_dev,
                         void* stream) {
  if (n_seqs < 0 || max_moves < 0) return FP4IDX_ERR_INVALID_ARG;
  const int st = check_pool(num_pages, max_pages, ratio, n_free, free_pages, pinned);
  if (st != FP4IDX_OK) return st;
  if (n_seqs > 65536 || max_moves > INT32_MAX) return FP4IDX_ERR_UNSUPPORTED;
  if (!counts || !workspace || (n_seqs > 0 && (!page_table || !cached_lens || !page_table_out))) return FP4IDX_ERR_INVALID_ARG;
  if (max_moves > 0 && (!move_src || !move_dst)) return FP4IDX_ERR_INVALID_ARG;
  if (n_seqs > 0 && page_table == page_table_out) return FP4IDX_ERR_INVALID_ARG;
  const void* ptrs[] = {page_table, cached_lens, page_table_out, move_src, move_dst, counts, status_dev};
  for (const void* p : ptrs)
    if (!aligned(p, 4)) return FP4IDX_ERR_INVALID_ARG;
  if (!aligned(workspace, 16)) return FP4IDX_ERR_INVALID_ARG;
  if (workspace_bytes < fp4idx_compact_pages_workspace_bytes(num_pages)) return FP4IDX_ERR_WORKSPACE;
  fp4idx::CompactArgs a{page_table, cached_lens, pinned, static_cast<int32_t*>(workspace), free_pages, page_table_out,
                        move_src, move_dst, counts, status_dev, (int32_t)n_seqs, max_pages, ratio, (int32_t)num_pages,
                        (int32_t)n_free, (int32_t)max_moves};
  return from_cuda(fp4idx::launch_compact_pages(a, as_stream(stream)));
}

}  // extern "C"
