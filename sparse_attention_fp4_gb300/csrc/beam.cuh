// Host launchers of the beam selection and of the page pool's operators, called by their C
// ABI (api_beam.cu).
#pragma once

#include "latent.cuh"

namespace fp4idx {

// What one chunk of a row's tokens leaves for the join: the largest logit, the sum of
// exp(logit - largest) as the sum of two floats, and how many candidates its list holds.
struct BeamStat {
  float top, sum, sum_low;
  int32_t count;
};
struct BeamItem {
  float logit;
  int32_t token;
};

// i / d by one product, for i and d below 2^16.
struct Divisor {
  int32_t d;
  uint32_t inverse;
  Divisor() = default;
  explicit Divisor(int32_t n) : d(n), inverse(n == 1 ? 0 : 0xFFFFFFFFu / n + 1) {}
#ifdef __CUDACC__
  __device__ int under(int i) const { return d == 1 ? i : (int)__umulhi((uint32_t)i, inverse); }
#endif
};

struct BeamArgs {
  const void* logits;
  const float* scores;
  const int32_t* done;
  float* out_scores;
  int32_t *out_rows, *out_tokens, *done_out, *status;
  BeamStat* stats;  // [n_rows, chunks]
  BeamItem* lists;  // [n_rows, chunks, k], each in descending order
  int64_t stride;
  int32_t n_rows, vocab, beams, k, end_token;
  int32_t chunks, chunk_vecs;  // chunks of a row, and how many 16-byte vectors of logits one has
  int32_t lanes;               // of a join, for a row's chunks
  Divisor by_k, by_beam, by_deep;  // a list's candidates, a row's, those of a list that make a join's bound
};
size_t beam_select_workspace_bytes(int64_t n_rows, int32_t vocab, int32_t k);
cudaError_t launch_beam_select(BeamArgs a, int32_t type, void* workspace, cudaStream_t stream);

struct ForkArgs {
  const int32_t *page_table, *cached, *parents;
  const uint32_t* pinned;
  int32_t* free_pages;
  const int32_t* free_head;
  int32_t *table_out, *cached_out, *copy_src, *copy_dst, *counts, *status;
  int32_t n_old, n_new, max_pages, ratio, num_pages, n_free;
};
cudaError_t launch_fork_pages(const ForkArgs& a, cudaStream_t stream);

struct CompactArgs {
  const int32_t *page_table, *cached;
  const uint32_t* pinned;
  int32_t* remap;  // [num_pages], written for every page in use from id counts[1] on, whether it moves or stays
  int32_t *free_pages, *table_out, *move_src, *move_dst, *counts, *status;
  int32_t n_seqs, max_pages, ratio, num_pages, n_free, max_moves;
};
cudaError_t launch_compact_pages(const CompactArgs& a, cudaStream_t stream);

// Caches of one call: passed by value with the launch.
struct Regions {
  uint8_t* base[FP4IDX_COPY_MAX_REGIONS];
  int32_t vecs[FP4IDX_COPY_MAX_REGIONS];  // 16-byte pieces of a page
  int32_t each[FP4IDX_COPY_MAX_REGIONS], first[FP4IDX_COPY_MAX_REGIONS];  // filled in by the launcher
  int32_t n;
};
cudaError_t launch_move_pages(const int32_t* src, const int32_t* dst, int64_t n_copies, const int32_t* count,
                              Regions& regions, int64_t num_pages, int32_t* status, cudaStream_t stream);

}  // namespace fp4idx
