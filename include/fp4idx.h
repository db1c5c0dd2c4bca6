/*
 * fp4idx.h -- C ABI of the GB300 FP4 indexer library (libfp4idx.so).
 *
 * The DeepSeek-V4 sparse-attention indexer, as described on three SGLang pull
 * request pages:
 *   [P1] "dsv4.1-amd: KV cache layouts, FP4 indexer, compressor and router kernels"
 *   [P2] "[AMD] Enable FP4 indexer for Deepseek V4"
 *   [P3] "[AMD] DeepSeek-V4.1-Flash on MI350X (gfx950)"
 * Write side: each compressed bf16 index-K row of 128 goes through RMSNorm, RoPE
 * (dims 0..63), a 128-point Hadamard rotation and e2m1 quantisation with one
 * UE8M0 scale per 32 elements, into a paged cache split into a 64-byte payload
 * tensor and a 4-byte scale tensor.  Read side: paged-MQA logits
 *   logits[t,s] = sum_h w[t,h] * ReLU(q_fp4[t,h] . k_fp4[s]),  s < context_lens[t],
 * then a per-row top-k of compressed-token indices, ascending.
 * Around the indexer: the step's maps built on the device (fp4idx_plan_step), and the cache
 * and attention that the selection is for (fp4idx_store_latent, fp4idx_latent_attn_topk,
 * fp4idx_latent_attn, fp4idx_latent_prefill).  For requests decoded as several hypotheses:
 * the choice of the hypotheses that go on (fp4idx_beam_select), and the page pool's care
 * (fp4idx_fork_pages, fp4idx_copy_pages, fp4idx_compact_pages).
 *
 * Conventions for every entry point
 *   - Pointers are DEVICE pointers (cudaMalloc / torch CUDA memory on the current
 *     device) unless marked "host".  Arrays are dense, row-major, 16-byte aligned.
 *   - bf16 values are passed as uint16_t bit patterns.
 *   - Ownership stays with the caller.  The library never allocates, frees or
 *     synchronises; every call only enqueues kernels on `stream` (a cudaStream_t,
 *     NULL = the legacy default stream) and returns.  Calls are safe inside CUDA
 *     graph capture.
 *   - Return value: FP4IDX_OK, or an fp4idx_status for a problem the host can see
 *     (null pointer, bad size, misalignment, unsupported shape, too small a
 *     workspace, a failed launch).  Nothing is enqueued when a call fails.
 *   - status_dev (nullable, one int32 in device memory, zero it before use): the
 *     kernels record the first data-dependent error they meet (a page id outside
 *     [0, num_pages), a slot past the cache, a position outside the RoPE table, a
 *     context length above the stated maximum, a pipeline wait that ran out).
 *     They skip the offending access and never trap.
 *   - Fixed shapes: head_dim 128, 64 indexer heads, 64 tokens per cache page.
 *   - Devices: calls run on the current device.  The first call of a kernel on each
 *     device sets that kernel's shared-memory size attribute there (once per device,
 *     thread-safe), so make the first call of each entry point on a device outside
 *     stream capture.
 *
 * Cache layout (split, [P2] Motivation): per physical page p and token j < 64,
 *   payload[p][c][j][0..15]  (uint8, [num_pages,4,64,16]; 64 B per token)
 *   scale  [p][c][j]         (uint8, [num_pages,4,64];    4 B per token)
 * c = 32-element block (element 32c+2b in the low nibble of byte b, 32c+2b+1 in
 * the high nibble), scale byte = e + 127 where the block is e2m1(x * 2^-e).
 * Slot of token j on page p: p*64 + j.
 * Query layout (this library's own, shaped like one K page with heads in place
 * of tokens): q_payload[t][c][h][0..15] ([T,4,64,16]), q_scale[t][c][h] ([T,4,64]).
 */
#ifndef FP4IDX_H
#define FP4IDX_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define FP4IDX_HEAD_DIM 128
#define FP4IDX_NUM_HEADS 64
#define FP4IDX_PAGE_TOKENS 64
#define FP4IDX_FP8_PAGE_BYTES (64 * 128 + 64 * 4)
#define FP4IDX_MAX_TOPK 4096
#define FP4IDX_MAX_CONTEXT 65536
#define FP4IDX_MAX_HIDDEN 16384 /* hidden size limit of fp4idx_quant_q_w */
#define FP4IDX_LATENT_VALUE 512  /* value dims of a latent row: its first 512 */
#define FP4IDX_LATENT_MAX_HEADS 128
#define FP4IDX_LATENT_MAX_ROWS (1 << 20)
#define FP4IDX_LATENT_MAX_TREE_WORDS 8 /* 256 drafted tokens a sequence */
#define FP4IDX_PREFILL_KEY 192   /* expanded attention: 128 dims of the head's own key, 64 shared rotated dims */
#define FP4IDX_PREFILL_VALUE 128
#define FP4IDX_BEAM_MAX_BEAMS 64
#define FP4IDX_BEAM_MAX_K 64
#define FP4IDX_BEAM_MAX_VOCAB (1 << 19)
#define FP4IDX_BEAM_MAX_ROWS (1 << 20)
#define FP4IDX_FORK_MAX_ROWS 8192           /* rows of a page table, old and new */
#define FP4IDX_MAX_POOL_PAGES (1 << 23)     /* fork and compaction: pages of a pool */
#define FP4IDX_COPY_MAX_REGIONS 256         /* caches of one fp4idx_copy_pages call */
#define FP4IDX_TOPK_NOALLOC_MAX_BYTES (16u * 1024u * 1024u) /* fixed scratch of fp4idx_topk_noalloc */

typedef enum {
  FP4IDX_OK = 0,
  FP4IDX_ERR_INVALID_ARG = 1,  /* null pointer, negative size, misaligned pointer, k out of range */
  FP4IDX_ERR_UNSUPPORTED = 2,  /* a shape the kernels do not implement (heads != 64, ...) */
  FP4IDX_ERR_CUDA = 3,         /* a CUDA launch or attribute call failed */
  FP4IDX_ERR_WORKSPACE = 4,    /* schedule/workspace buffer smaller than the size query says */
  FP4IDX_ERR_BAD_PAGE = 5,     /* device: page id / slot outside the cache */
  FP4IDX_ERR_TIMEOUT = 6,      /* device: a pipeline wait exceeded its iteration limit */
  FP4IDX_ERR_BAD_POSITION = 7, /* device: RoPE position outside [0, max_pos) */
  FP4IDX_ERR_BAD_LENGTH = 8,   /* device: context length < 0 or above max_context / page-table width */
  FP4IDX_ERR_SCHEDULE = 9,     /* schedule built for another row count or grid, or its selection
                                  counters were left non-zero by a call that failed: rebuild it */
  FP4IDX_ERR_SCRATCH_LIMIT = 10, /* fp4idx_topk_noalloc: the call needs more than its fixed scratch */
  FP4IDX_ERR_CAPACITY = 11,      /* device: a plan or a fork ran out of rows, stores or free pages, or a free
                                    list of room */
  FP4IDX_ERR_BAD_VALUE = 12      /* device: fp4idx_beam_select met a NaN or +inf */
} fp4idx_status;

/* Human-readable name of a status code (static string). */
const char* fp4idx_status_string(int status);

/* Number of SMs of the current device (host out-pointer). */
int fp4idx_num_sms(int32_t* num_sms_out);

/*
 * K store -- the fused writer of [P2] Modifications / FP4 kernel adapters
 * ("fused RMSNorm, RoPE, Hadamard, FP4 quantization, and paged cache writes")
 * into the split layout of [P2] Motivation; round-to-nearest-even per [P1] Summary.
 *   k          [n_rows,128] bf16   compressed index-K rows
 *   positions  [n_rows] int32      RoPE position of each row, in [0, max_pos)
 *   slots      [n_rows] int32      destination slot page*64+j; slot < 0 = padding, skipped
 *   norm_w     [128] bf16          RMSNorm weight ([P2] compressor.py BF16 mirror)
 *   eps                            RMSNorm epsilon (1e-6 for DeepSeek-V4)
 *   cos_sin    [max_pos,64] bf16   row p: cos(p f_i) for i<32, then sin(p f_i)
 *   payload    [num_pages,4,64,16] uint8, scale [num_pages,4,64] uint8 (written)
 * Device errors: BAD_PAGE (slot >= num_pages*64), BAD_POSITION; the row is skipped.
 */
int fp4idx_store_k(const uint16_t* k, int64_t n_rows, const int32_t* positions, const int32_t* slots,
                   const uint16_t* norm_w, float eps, const uint16_t* cos_sin, int32_t max_pos,
                   uint8_t* payload, uint8_t* scale, int64_t num_pages, int32_t* status_dev, void* stream);

/*
 * K store into the FP8 "fused" indexer layout, 132 bytes per token ([P2] Device
 * memory and sizing: the FP8 footprint the FP4 entry replaces).  Same chain up to
 * the Hadamard, then one fp32 scale per token s = amax/448 (1 if amax = 0) and
 * e4m3 = RNE-satfinite(x / s).  Page layout (fp8_pages, [num_pages, 8448] uint8):
 * bytes [j*128, j*128+128) = token j's e4m3 values, bytes [8192 + 4j, 8192 + 4j + 4)
 * = its fp32 scale.  Arguments and errors as fp4idx_store_k.
 */
int fp4idx_store_k_fp8(const uint16_t* k, int64_t n_rows, const int32_t* positions, const int32_t* slots,
                       const uint16_t* norm_w, float eps, const uint16_t* cos_sin, int32_t max_pos,
                       uint8_t* fp8_pages, int64_t num_pages, int32_t* status_dev, void* stream);

/*
 * Q quant -- [P2] Modifications / fp4_indexer_hip.py "Q RoPE/Hadamard/FP4
 * quantization" and [P1] Summary's query packer: RoPE at q_positions[t], Hadamard,
 * e2m1 + UE8M0/32.  No RMSNorm on the query side.
 *   q [n_rows, n_heads, 128] bf16;  q_positions [n_rows] int32
 *   q_payload [n_rows,4,64,16] uint8, q_scale [n_rows,4,64] uint8 (written)
 * n_heads must be 64 (UNSUPPORTED otherwise).  Device error: BAD_POSITION.
 */
int fp4idx_quant_q(const uint16_t* q, int64_t n_rows, int32_t n_heads, const int32_t* q_positions,
                   const uint16_t* cos_sin, int32_t max_pos, uint8_t* q_payload, uint8_t* q_scale,
                   int32_t* status_dev, void* stream);

/*
 * FP8 query pack -- the query side of the FP8 comparison path ([P2] Device memory and
 * sizing: the 132 B/token FP8 entry the FP4 entry replaces).  RoPE and the Hadamard as in
 * fp4idx_quant_q, then the K side's FP8 rule per (row, head): s = amax/448 (1 if amax = 0),
 * e4m3 = RNE-satfinite(x / s).  The pages give only the K entry; this rule for the query is
 * a reading.
 *   q8 [n_rows,8,64,16] uint8: q8[t][c][h][i] = element 16c + i of head h (written)
 *   q8_scale [n_rows,64] fp32 (written)
 * n_heads must be 64.  Device error: BAD_POSITION.
 */
int fp4idx_quant_q_fp8(const uint16_t* q, int64_t n_rows, int32_t n_heads, const int32_t* q_positions,
                       const uint16_t* cos_sin, int32_t max_pos, uint8_t* q8, float* q8_scale, int32_t* status_dev,
                       void* stream);

/*
 * Q quant and head weights in one launch -- [P1] Summary: "a one-launch index-Q pack +
 * head weights", where indexer_head_weights runs a batch-invariant split-K bf16 GEMV whose
 * result stays in fp32.  The queries are packed exactly as fp4idx_quant_q packs them
 * (same arguments, same bytes); beside them
 *   w_out[t][h] = w_scale * sum_d hidden[t][d] * w_proj[h][d]      (fp32, [n_rows, 64])
 *   hidden [n_rows, hidden_dim] bf16; w_proj [64, hidden_dim] bf16 (row h: head h)
 *   hidden_dim a multiple of 256, at most FP4IDX_MAX_HIDDEN (UNSUPPORTED otherwise)
 * The pages give neither the hidden size nor a scale: any constant factor goes into
 * w_scale.  Order of the sum (the same for every batch, so a row's weights do not depend
 * on the rows beside it): the hidden dimension is cut into M = hidden_dim/256 chunks of
 * 256 and the chunks into 8 runs [wM/8, (w+1)M/8); in run w, lane l of 32 adds the products
 * d = 256m + 8l + i, m then i ascending, one fp32 rounding per addition (bf16 products are
 * exact in fp32); then the 32 lane sums pairwise at lane distances 16, 8, 4, 2, 1; then the
 * 8 run sums in run order; then one rounding for w_scale.  A product meets at most
 * 8*ceil(M/8) + 12 <= hidden_dim/256 + 19 roundings, so the result is within
 * (hidden_dim/256 + 20) * 2^-24 * |w_scale| * sum_d |hidden*w_proj| of the exact value.
 */
int fp4idx_quant_q_w(const uint16_t* q, int64_t n_rows, int32_t n_heads, const int32_t* q_positions,
                     const uint16_t* cos_sin, int32_t max_pos, const uint16_t* hidden, int32_t hidden_dim,
                     const uint16_t* w_proj, float w_scale, uint8_t* q_payload, uint8_t* q_scale, float* w_out,
                     int32_t* status_dev, void* stream);

/*
 * Schedule -- the length-balanced split of the logits work over the GPU
 * ([P1] Summary: an in-tree decode schedule whose registers do not grow with the
 * row count; [P2] Attention runtime: schedules built during graph capture and
 * reused across all C4 layers of a forward).  One small device kernel: no host
 * sync, capturable, a pure function of (context_lens, row_seq, n_rows, num_ctas),
 * so a schedule built once serves every layer of the same batch.
 *   context_lens [n_rows] int32  visible compressed tokens of each query row
 *                                (padded rows: 0; prefill rows: floor((p+1)/4))
 *   row_seq      [n_rows] int32  sequence (page-table row) of each query row; rows
 *                                of one sequence that are adjacent share K tiles
 *   num_ctas                     grid the logits kernel will use (0 = SM count)
 *   schedule     device buffer of at least fp4idx_schedule_workspace_bytes(n_rows, num_ctas)
 * Besides the work split, the schedule holds one counter per row that the fused
 * selection of fp4idx_logits_topk_fused counts up and puts back to zero; the build
 * zeroes them.
 */
size_t fp4idx_schedule_workspace_bytes(int64_t max_rows, int32_t num_ctas);
int fp4idx_build_schedule(const int32_t* context_lens, const int32_t* row_seq, int64_t n_rows,
                          int32_t num_ctas, void* schedule, size_t schedule_bytes, void* stream);

/*
 * The decode step's preparation in one launch: the work of fp4idx_build_schedule,
 * fp4idx_store_k and fp4idx_quant_q, with the same arguments and the same results
 * (bit for bit), in one grid -- [P2] Attention runtime (the schedule is built in the
 * captured step) and Modifications (the fused K writer and the Q packer).  One block builds
 * the schedule, the others store the n_new K rows and pack the n_rows query rows; they
 * run side by side, and the whole grid allows the logits launch that follows on the
 * stream (fp4idx_logits_topk, fp4idx_logits) to start its own set-up before the grid ends.
 * Arguments as in the three calls; q_positions, context_lens and row_seq describe the
 * n_rows query rows, k, positions and slots the n_new K rows (n_new may be 0).
 * Device errors: those of the three calls.
 */
int fp4idx_prepare_step(const uint16_t* k, int64_t n_new, const int32_t* positions, const int32_t* slots,
                        const uint16_t* norm_w, float eps, const uint16_t* q, int64_t n_rows, int32_t n_heads,
                        const int32_t* q_positions, const uint16_t* cos_sin, int32_t max_pos, uint8_t* payload,
                        uint8_t* scale, int64_t num_pages, uint8_t* q_payload, uint8_t* q_scale,
                        const int32_t* context_lens, const int32_t* row_seq, int32_t num_ctas, void* schedule,
                        size_t schedule_bytes, int32_t* status_dev, void* stream);

/*
 * Paged-MQA logits + top-k -- [P2] Modifications: "Dispatch decode and prefill
 * FP4 paged-MQA logits" over the split cache through a guarded page table; padded
 * rows keep context length 0 ([P2] Attention runtime); the selection is sorted
 * and ordered by position ([P3] Changes, Historical results).
 *   q_payload/q_scale   output of fp4idx_quant_q for the n_rows rows
 *   w                   [n_rows,64] fp32 head weights
 *   payload/scale       the split K cache, num_pages pages
 *   page_table          [num_seqs, max_pages] int32 physical page of logical page i
 *   row_seq, context_lens  as given to fp4idx_build_schedule (same arrays)
 *   max_context         host-known upper bound of context_lens (<= FP4IDX_MAX_CONTEXT)
 *   k                   1..FP4IDX_MAX_TOPK
 *   schedule            built by fp4idx_build_schedule for these rows (read only here)
 *   workspace           >= fp4idx_logits_workspace_bytes(n_rows, max_context, k) bytes:
 *                       a logits buffer (unused when logits_out is given) and the
 *                       selection's scratch; nothing in it needs to be initialised
 *   topk_idx  [n_rows,k] int32 (written): the k highest-logit token indices of each
 *             row in ascending order; all of them when context_len <= k; -1 pads.
 *   logits_out [n_rows, logits_stride] fp32 (nullable): when given, receives
 *             logits[t,s] for s < context_lens[t] (the rest is not written).
 * Two launches: the logits kernel, then the top-k kernel (one CTA, or a pair of CTAs
 * in a cluster, per row).
 * Device errors: BAD_PAGE (page id out of range: the tile is skipped),
 * BAD_LENGTH, TIMEOUT, SCHEDULE.
 */
size_t fp4idx_logits_workspace_bytes(int64_t max_rows, int32_t max_context, int32_t k);
int fp4idx_logits_topk(const uint8_t* q_payload, const uint8_t* q_scale, const float* w, int64_t n_rows,
                       int32_t n_heads, const uint8_t* payload, const uint8_t* scale, int64_t num_pages,
                       const int32_t* page_table, int64_t num_seqs, int32_t max_pages, const int32_t* row_seq,
                       const int32_t* context_lens, int32_t max_context, int32_t k, const void* schedule,
                       size_t schedule_bytes, void* workspace, size_t workspace_bytes, int32_t* topk_idx,
                       float* logits_out, int64_t logits_stride, int32_t* status_dev, void* stream);

/*
 * fp4idx_logits_topk in one launch ([P3] Changes: "sorted top-k selection"; the
 * selection is folded into the logits kernel).  Same arguments, result and errors, with
 * one difference: `schedule` is written.  When n_rows is at most the device's SM count,
 * the epilogue warps count, per row, the pieces of its logits they have written (a
 * release add on a counter in the schedule); after its own work the CTA of each row --
 * or a pair of CTAs in a cluster, when the grid holds two for every row -- waits for all
 * of the row's pieces (bounded) and selects the row from the logits in L2.  The launch
 * is cooperative (every CTA resident at once).  The counters go back to zero, so calls
 * that share a schedule must be ordered (one stream), and after a call that reported an
 * error the schedule must be built again.  Larger batches run the two launches of
 * fp4idx_logits_topk.  Both give the same selection.  Inside a CUDA graph, where the
 * second launch of fp4idx_logits_topk costs little, that call is the faster of the two on
 * GB300; this one saves the launch where launches are not overlapped.
 */
int fp4idx_logits_topk_fused(const uint8_t* q_payload, const uint8_t* q_scale, const float* w, int64_t n_rows,
                             int32_t n_heads, const uint8_t* payload, const uint8_t* scale, int64_t num_pages,
                             const int32_t* page_table, int64_t num_seqs, int32_t max_pages, const int32_t* row_seq,
                             const int32_t* context_lens, int32_t max_context, int32_t k, void* schedule,
                             size_t schedule_bytes, void* workspace, size_t workspace_bytes, int32_t* topk_idx,
                             float* logits_out, int64_t logits_stride, int32_t* status_dev, void* stream);

/*
 * The two halves of fp4idx_logits_topk, for callers that want the logits themselves or
 * select elsewhere.  fp4idx_logits writes logits_out[t][s] for s < context_lens[t]
 * (logits_stride >= max_context; the rest of each row is not written).  fp4idx_topk
 * selects from such a buffer: topk_idx[t] = the k largest of logits[t][0..L_t), ascending
 * positions, -1 padding; ties at the k-th value go to the lower positions.  Its scratch
 * (per row, the sort keys of the positions past the first 32,768, which do not fit in
 * shared memory; at least 256 bytes even when max_context <= 32768) lives in `workspace`,
 * at least fp4idx_topk_workspace_bytes(n_rows, max_context) bytes, 16-byte aligned;
 * nothing in it needs to be initialised.
 */
int fp4idx_logits(const uint8_t* q_payload, const uint8_t* q_scale, const float* w, int64_t n_rows, int32_t n_heads,
                  const uint8_t* payload, const uint8_t* scale, int64_t num_pages, const int32_t* page_table,
                  int64_t num_seqs, int32_t max_pages, const int32_t* row_seq, const int32_t* context_lens,
                  int32_t max_context, const void* schedule, size_t schedule_bytes, float* logits_out,
                  int64_t logits_stride, int32_t* status_dev, void* stream);
size_t fp4idx_topk_workspace_bytes(int64_t max_rows, int32_t max_context);
int fp4idx_topk(const float* logits, int64_t logits_stride, const int32_t* context_lens, int64_t n_rows,
                int32_t max_context, int32_t k, void* workspace, size_t workspace_bytes, int32_t* topk_idx,
                int32_t* status_dev, void* stream);

/*
 * FP8 logits -- the read side of the FP8 comparison path ([P2] Device memory and sizing:
 * the fused 132 B/token FP8 entry that the 68 B FP4 entry replaces), over the pages of
 * fp4idx_store_k_fp8 and the queries of fp4idx_quant_q_fp8:
 *   logits[t,s] = sum_h w[t,h] * ReLU(q[t,h] . k[s]),  s < context_lens[t],
 * with q = e4m3(q8[t,.,h,.]) * q8_scale[t,h] and k = e4m3(token s's 128 bytes) * its fp32
 * scale.  Tensor-core kernel (e4m3 x e4m3 -> f32); the two scales are applied in fp32
 * after the dot products.
 *   q8 [n_rows,8,64,16] uint8, q8_scale [n_rows,64] fp32, w [n_rows,64] fp32
 *   fp8_pages [num_pages, 8448] uint8 (1 <= num_pages <= INT32_MAX)
 *   page_table, row_seq, context_lens, max_context, schedule: as fp4idx_logits (the same
 *   schedule serves both formats)
 *   logits_out [n_rows, logits_stride] fp32: written for s < context_lens[t], NaN where
 *   the token's page id is out of range; the rest of each row is not written.
 * All pointers 16-byte aligned except page_table, row_seq, context_lens, logits_out and
 * status_dev (4-byte).  Device errors: BAD_PAGE, BAD_LENGTH, TIMEOUT, SCHEDULE.
 */
int fp4idx_logits_fp8(const uint8_t* q8, const float* q8_scale, const float* w, int64_t n_rows, int32_t n_heads,
                      const uint8_t* fp8_pages, int64_t num_pages, const int32_t* page_table, int64_t num_seqs,
                      int32_t max_pages, const int32_t* row_seq, const int32_t* context_lens, int32_t max_context,
                      const void* schedule, size_t schedule_bytes, float* logits_out, int64_t logits_stride,
                      int32_t* status_dev, void* stream);

/*
 * FP8 logits + top-k in one call: fp4idx_logits_fp8 into a logits buffer, then the
 * selection of fp4idx_topk.  Workspace, k, topk_idx and logits_out (nullable) as in
 * fp4idx_logits_topk; the other arguments as in fp4idx_logits_fp8.  A token on an
 * out-of-range page has a NaN logit (status BAD_PAGE), and its place in the selection is
 * then unspecified.
 */
int fp4idx_logits_topk_fp8(const uint8_t* q8, const float* q8_scale, const float* w, int64_t n_rows, int32_t n_heads,
                           const uint8_t* fp8_pages, int64_t num_pages, const int32_t* page_table, int64_t num_seqs,
                           int32_t max_pages, const int32_t* row_seq, const int32_t* context_lens,
                           int32_t max_context, int32_t k, const void* schedule, size_t schedule_bytes,
                           void* workspace, size_t workspace_bytes, int32_t* topk_idx, float* logits_out,
                           int64_t logits_stride, int32_t* status_dev, void* stream);

/*
 * fp4idx_topk_noalloc -- fp4idx_topk for callers that may not allocate device memory.
 * The pages this library follows have no counterpart: it is an interface addition.
 * A serving runtime that gives all of its memory to its own pool at start-up, or a
 * plug-in host that passes a library only a stream and the call's tensors, cannot hand
 * fp4idx_topk a workspace; this entry point takes none.
 *
 * Same arguments and result as fp4idx_topk, without workspace/workspace_bytes.  The
 * top-k scratch is a fixed array of the library's device code,
 * FP4IDX_TOPK_NOALLOC_MAX_BYTES per device; no call allocates or frees anything
 * itself (but see the set-up below).
 *   - Limit: fp4idx_topk_workspace_bytes(n_rows, max_context) must not exceed
 *     FP4IDX_TOPK_NOALLOC_MAX_BYTES (any row count fits at max_context <= 32768, up to
 *     128 rows at 65536); a larger call returns FP4IDX_ERR_SCRATCH_LIMIT and enqueues
 *     nothing.
 *   - Setup: the first valid call on each device (with that device current) looks up
 *     the array's address once.  Under CUDA's default lazy module loading that is also
 *     when the array's memory is committed on the device, so the first call can fail
 *     for lack of memory and may synchronise: make it at start-up, before a memory pool
 *     reserves the device's memory and before any stream capture begins.  A call with
 *     n_rows = 0 (other pointers may then be null) does the set-up and nothing else.
 *     Argument errors are reported before the set-up is attempted.  The address is
 *     kept for the life of the process; after cudaDeviceReset the entry point must not
 *     be used on that device again.  Of the conventions at the top of this file, the
 *     one on graph capture is not stated for this entry point.
 *   - Nothing in the array needs to start at zero: a call writes every key it
 *     reads back.
 *   - All calls on a device share the array: calls whose kernels may overlap (unordered
 *     streams, concurrent host threads) race on it.  Order them on one stream.
 */
int fp4idx_topk_noalloc(const float* logits, int64_t logits_stride, const int32_t* context_lens, int64_t n_rows,
                        int32_t max_context, int32_t k, int32_t* topk_idx, int32_t* status_dev, void* stream);

/*
 * Whole pages of the split cache -- [P1] Summary (dequantize_k_cache_paged serves the
 * V4.1 layouts) and [P2] Device memory and sizing / HiCache integration (page-row views
 * of the separately allocated payload and scale buffers; FP4 indexer rows move to and
 * from host memory as whole pages, payload and scale as separate regions).
 *   page_ids  [n_pages] int32  pages to process; an id < 0 is padding (skipped, its
 *                              output untouched); an id >= num_pages records BAD_PAGE
 *                              in status_dev and is skipped.
 * fp4idx_dequant_pages: out [n_pages,64,128] fp32 (written), out[i][j][d] = the
 *   e2m1 value of element d of token j of page page_ids[i] times 2^(scale byte - 127),
 *   exact in fp32 (values past the fp32 range, possible only for scale bytes >= 253,
 *   become +-inf).
 * fp4idx_export_pages: rows_payload [n_pages,4096] uint8 and rows_scale [n_pages,256]
 *   uint8 (written) = the payload and scale bytes of page page_ids[i], unchanged: page
 *   rows ready for one host copy each region.
 * fp4idx_import_pages: the reverse, writing page page_ids[i] of payload/scale from row
 *   i.  The ids of one call must be distinct (two rows into one page race).
 * rows_* and out are 16-byte aligned device buffers owned by the caller.
 */
int fp4idx_dequant_pages(const uint8_t* payload, const uint8_t* scale, int64_t num_pages, const int32_t* page_ids,
                         int64_t n_pages, float* out, int32_t* status_dev, void* stream);
int fp4idx_export_pages(const uint8_t* payload, const uint8_t* scale, int64_t num_pages, const int32_t* page_ids,
                        int64_t n_pages, uint8_t* rows_payload, uint8_t* rows_scale, int32_t* status_dev,
                        void* stream);
int fp4idx_import_pages(const uint8_t* rows_payload, const uint8_t* rows_scale, const int32_t* page_ids,
                        int64_t n_pages, uint8_t* payload, uint8_t* scale, int64_t num_pages, int32_t* status_dev,
                        void* stream);

/*
 * Context-parallel top-k -- [P3] the context-parallel runs (one long sequence's
 * compressed tokens sharded over GPUs): each shard scores its own token range and keeps
 * its top-k; the row's selection is the top-k of the gathered (value, index)
 * candidates.  The merge is exact: every token of the row's top-k is in its shard's
 * top-k, ties included (both sides give equal values to the lower position).
 * fp4idx_topk_values: values[t][i] = logits[t][topk_idx[t][i]] (the values of a
 *   selection made by fp4idx_topk on the same buffer); -inf where topk_idx is -1.
 *   n_rows <= 65535.
 * fp4idx_topk_merge: cand_values/cand_idx [n_rows, n_shards, k] fp32/int32: per row and
 *   shard, the shard's selection as GLOBAL positions (ascending, -1 padding at the end)
 *   with their values; shards in ascending position order (every position of shard s
 *   below every position of shard s+1).  topk_idx [n_rows, k] (written): the k largest
 *   candidates of the row, equal values to the lower position, ascending, -1 padding --
 *   the same selection fp4idx_topk makes on the whole row.  n_shards * k <=
 *   FP4IDX_MAX_CONTEXT, n_shards <= 1024, n_rows <= 65535; workspace of at least
 *   fp4idx_topk_merge_workspace_bytes(n_rows, n_shards, k) bytes, 16-byte aligned,
 *   nothing in it needs to be initialised.  Device errors as fp4idx_topk.
 */
size_t fp4idx_topk_merge_workspace_bytes(int64_t max_rows, int32_t n_shards, int32_t k);
int fp4idx_topk_values(const float* logits, int64_t logits_stride, const int32_t* topk_idx, int64_t n_rows, int32_t k,
                       float* values, void* stream);
int fp4idx_topk_merge(const float* cand_values, const int32_t* cand_idx, int64_t n_rows, int32_t n_shards, int32_t k,
                      void* workspace, size_t workspace_bytes, int32_t* topk_idx, int32_t* status_dev, void* stream);

/*
 * Step plan -- the maps that the other entry points take, built on the device from
 * request lengths: page table, cache slots, row positions, row sequences, context
 * lengths.  The pages build them on the host (prefill rows: floor((p+1)/4)); this is an
 * interface addition, so that a captured step needs no host work.
 * Sequence b has c = cached_lens[b] tokens and gets n = new_lens[b] more.  One cache
 * entry stands for `ratio` tokens (4 for the compressed index keys, 1 for one entry a
 * token): floor(c/ratio) entries exist, those up to floor((c+n)/ratio) are stored by
 * this step.
 *   cached_lens, new_lens [n_seqs] int32, n_seqs <= 65536; ratio 1..64
 *   free_pages [n_free] int32  page ids to take, from index *free_head on (free_head:
 *                              device int32, nullable = 0); n_free may be 0
 *   page_table [n_seqs, max_pages] int32 (read, and written where a sequence grows):
 *              holds the pages of the entries that exist; pages for the new entries are
 *              taken in sequence order and written behind them
 *   q_positions, row_seq, context_lens [max_rows] int32 (written): row i of the step is
 *              a new token of sequence row_seq[i] at position p = c + (its index among
 *              the new tokens), context length floor((p+1)/ratio).  Rows behind the last
 *              one: position 0, sequence 0, context length 0 (padding).
 *   store_positions, store_slots [max_stores] int32 (written): per new entry its index
 *              in the sequence and its slot page*64 + j; behind the last one 0 and -1
 *              (padding, skipped by the store kernels).
 *   cu_rows, cu_context [n_seqs+1] int32 (written): offsets of the sequences' rows, and
 *              of their entries after the step, each packed in sequence order
 *   counts [4] int32 (written): rows, stores, pages taken, sequences planned
 *   max_rows, max_stores <= 2^30
 * *free_head and cached_lens are not written: the caller adds counts[2] and new_lens
 * when the step is done (a repeated call gives the same result).
 * Sequences are planned in order; the first whose rows, stores or pages do not fit in
 * max_rows, max_stores or the free pages, or with whom cu_context would pass 2^31-1, and
 * all behind it, get no rows, pages or context (CAPACITY).  A sequence with a negative
 * length, or more entries than 64*max_pages, gets none either (BAD_LENGTH); those behind
 * it are planned.  An entry whose page id is negative or above 2^25-1 gets slot -1
 * (BAD_PAGE).  The outputs must not overlap one another or the inputs.  All pointers
 * 4-byte aligned.
 */
int fp4idx_plan_step(const int32_t* cached_lens, const int32_t* new_lens, int64_t n_seqs, int32_t ratio,
                     const int32_t* free_pages, int64_t n_free, const int32_t* free_head, int32_t* page_table,
                     int32_t max_pages, int32_t* q_positions, int32_t* row_seq, int32_t* context_lens,
                     int64_t max_rows, int32_t* store_positions, int32_t* store_slots, int64_t max_stores,
                     int32_t* cu_rows, int32_t* cu_context, int32_t* counts, int32_t* status_dev, void* stream);

/*
 * Latent store -- the write side of the cache that the attention behind the indexer
 * reads.  A latent row has `width` (512 or 576) bf16 values; all of them are the key of
 * its token, the first 512 its value, shared by all heads.
 *   kv         [n_rows, width] bf16
 *   positions, slots, eps, cos_sin, max_pos  as fp4idx_store_k
 *   norm_w     [512] bf16
 *   cache      [num_pages, 64, width] bf16 (written): token j of page p at slot p*64 + j
 * Row: y = x * rsqrt(mean(x^2 over dims 0..511) + eps) * norm_w on dims 0..511, then
 * RoPE on the last 64 dims, pairs (i, i+32) as in the index keys (width 512: the
 * normalised dims 448..511; width 576: dims 512..575, which are not normalised).  fp32
 * throughout, rounded to bf16 once.
 * Device errors: BAD_PAGE, BAD_POSITION; the row is skipped.  TIMEOUT: rows may be missing
 * from the cache.  Slots of one call must be distinct.
 */
int fp4idx_store_latent(const uint16_t* kv, int64_t n_rows, int32_t width, const int32_t* positions,
                        const int32_t* slots, const uint16_t* norm_w, float eps, const uint16_t* cos_sin,
                        int32_t max_pos, uint16_t* cache, int64_t num_pages, int32_t* status_dev, void* stream);

/*
 * Absorbed latent attention over a selection of tokens -- what the selection of
 * fp4idx_logits_topk is for:
 *   s[h,i] = scale * q[t,h,:] . k[topk_idx[t,i],:]       (key: all `width` dims)
 *   out[t,h,:] = sum_i softmax_i(s[h,i]) k[topk_idx[t,i], 0..511]
 *   lse[t,h]   = log sum_i exp(s[h,i])
 *   q          [n_rows, n_heads, width] bf16, queries in latent space; n_heads 1..128
 *   cache      [num_pages, 64, width] bf16; page_table [num_seqs, max_pages], row_seq as above
 *   topk_idx   [n_rows, k] int32 token positions of the row's sequence; entries < 0 are
 *              skipped; a position listed twice counts twice
 *   context_lens [n_rows] int32, nullable: when given, only the first
 *              min(k, context_lens[t]) entries of the row are read (those that
 *              fp4idx_topk fills); negative counts as 0
 *   out        [n_rows, n_heads, 512] bf16 (written); lse [n_rows, n_heads] fp32 (nullable)
 * A row with no token gets out = 0 and lse = -inf.  Only listed tokens are read: what the
 * rest of the cache holds (NaN included) does not matter.  Scores, softmax and sums are
 * fp32; the weights are rounded to bf16 for the second product, the output once.
 * workspace: fp4idx_latent_attn_workspace_bytes(n_rows, n_heads) bytes, 16-byte aligned,
 * nothing in it needs to be initialised; calls that may overlap need one each.
 * Device errors: BAD_PAGE (row_seq outside [0, num_seqs), a position's page id outside
 * the cache), BAD_LENGTH (a position >= 64*max_pages); the token (the row for row_seq) is
 * skipped.  TIMEOUT: outputs are then not valid.
 */
size_t fp4idx_latent_attn_workspace_bytes(int64_t max_rows, int32_t n_heads);
int fp4idx_latent_attn_topk(const uint16_t* q, int64_t n_rows, int32_t n_heads, int32_t width, const uint16_t* cache,
                            int64_t num_pages, const int32_t* page_table, int64_t num_seqs, int32_t max_pages,
                            const int32_t* row_seq, const int32_t* topk_idx, int32_t k, const int32_t* context_lens,
                            float scale, void* workspace, size_t workspace_bytes, uint16_t* out, float* lse,
                            int32_t* status_dev, void* stream);

/*
 * Absorbed latent attention over the whole context, with an optional tree of drafted
 * tokens: as fp4idx_latent_attn_topk over the tokens s < context_lens[t] of the row's
 * sequence and, where tree_mask is given, the tokens context_lens[t] + j whose bit j of
 * the row's mask is set (bit j of word j/32; a drafted token's own bit and those of the
 * tokens above it in the tree).
 *   context_lens [n_rows] int32; max_context: host-known upper bound of
 *              context_lens[t] + (highest set bit + 1), at most 64*max_pages
 *   tree_mask  [n_rows, mask_words] uint32 bit patterns (nullable with mask_words 0),
 *              mask_words <= FP4IDX_LATENT_MAX_TREE_WORDS
 * Adjacent rows of one sequence share the reads of the cache when their heads fit one
 * pass together (n_heads <= 32).  Device errors as above; BAD_LENGTH (a context length
 * < 0, or one past max_context, drafted tokens included): the row has no token.
 */
int fp4idx_latent_attn(const uint16_t* q, int64_t n_rows, int32_t n_heads, int32_t width, const uint16_t* cache,
                       int64_t num_pages, const int32_t* page_table, int64_t num_seqs, int32_t max_pages,
                       const int32_t* row_seq, const int32_t* context_lens, int32_t max_context,
                       const uint32_t* tree_mask, int32_t mask_words, float scale, void* workspace,
                       size_t workspace_bytes, uint16_t* out, float* lse, int32_t* status_dev, void* stream);

/*
 * Expanded latent attention -- prompts, where each head's keys and values have been
 * expanded from the latent rows (the cheaper form while the context is shorter than the
 * selection).  Causal, over packed sequences:
 *   s[i,j,h] = scale * (q[i,h,0..127] . kv[j,h,0..127] + q[i,h,128..191] . k_rope[j,:])
 *   out[i,h,:] = sum_j softmax_j(s[i,j,h]) kv[j,h,128..255],  lse as above
 *   q      [n_q, n_heads, 192] bf16;  kv [n_kv, n_heads, 256] bf16 (128 key dims, then 128
 *          value dims);  k_rope [n_kv, 64] bf16, shared by the heads;  n_heads 1..1024
 *   cu_q, cu_kv [n_seqs+1] int32  offsets of the sequences' rows, non-decreasing from >= 0;
 *          query i of a sequence with nq queries and nkv keys sees its keys
 *          j <= nkv - nq + i (the queries are the last nq tokens); none where that is < 0
 *   max_q, max_kv  host-known upper bounds of a sequence's queries and keys
 *   out    [n_q, n_heads, 128] bf16, lse [n_q, n_heads] fp32 (nullable): written for the
 *          rows of sequences only (rows from cu_q[n_seqs] on are left as they were)
 * A row that sees no key gets out = 0 and lse = -inf.  Keys and values behind a
 * sequence's end do not matter (NaN included); within a sequence a non-finite value row
 * may also reach the up to 255 query rows before it.  fp32 scores, softmax and sums; the
 * weights are rounded to bf16 for the second product, the output once.
 * Device errors: BAD_LENGTH (offsets that decrease, leave the arrays or exceed max_q /
 * max_kv: the sequence is skipped).  TIMEOUT: outputs are then not valid.
 */
int fp4idx_latent_prefill(const uint16_t* q, int64_t n_q, int32_t n_heads, const uint16_t* kv, int64_t n_kv,
                          const uint16_t* k_rope, const int32_t* cu_q, const int32_t* cu_kv, int64_t n_seqs,
                          int32_t max_q, int32_t max_kv, float scale, uint16_t* out, float* lse, int32_t* status_dev,
                          void* stream);

/*
 * Beam selection -- the hypotheses of a request that go on, over its beams and the
 * vocabulary.  The pages stop at the attention; this and the page operators below are
 * interface additions for requests that are decoded as several hypotheses.
 * Rows g*n_beams .. g*n_beams + n_beams - 1 are the beams of group (request) g:
 *   total[r,v] = scores[r] + (logits[r,v] - log sum_u exp(logits[r,u]))
 * and a finished row (done[r] != 0) has the one candidate (end_token, scores[r]); its
 * logits are not read.  Per group the k largest totals, in descending order; of equal
 * totals the lower row comes first, then the lower token.
 *   logits      [n_rows, vocab] of type logits_type (0 bf16, 1 fp16, 2 fp32), row r at
 *               element r*logits_stride; aligned to its element type; a token is ruled out
 *               by -inf
 *   scores      [n_rows] fp32, the rows' scores so far; -inf: the row is dead (no
 *               candidate, its logits are not read)
 *   n_rows a multiple of n_beams, n_beams 1..64, k 1..64, vocab 1..2^19
 *   done        [n_rows] int32, nullable (with it, end_token is a token of the vocabulary)
 *   end_token   -1: none
 *   out_scores, out_rows, out_tokens [n_rows/n_beams, k] (written): total (fp32), row (of
 *               all n_rows: the parents of fp4idx_fork_pages) and token; -inf, -1 and -1
 *               where a group has no candidate left
 *   done_out    [n_rows/n_beams, k] int32, nullable (written): 1 where the row was finished
 *               or the token is end_token, else 0
 * The logarithm of a row's sum is off by less than (30 + 6 t + 2.3 ln(vocab)) * 2^-24, however
 * small it is itself, where t is vocab/2048 for fp32 and vocab/4096 for 16-bit logits, rounded
 * up, 64 at the most (2.7e-5 for the longest rows; 1e-7 is usual, 6e-7 the most that was seen):
 * exponentials, a thread's share of their sum and the factors between shares are fp32.  What is
 * added up above that, and the totals, has some 36 bits or more.  Totals of different rows
 * closer than twice that error may change places; within a row the order is that of the logits
 * (but for logits of one row so close that their totals agree to 36 bits).  A total below
 * fp32's range is written as -inf, with its row and token.  A row whose score or logits hold a
 * NaN or +inf has no candidate (BAD_VALUE).  The outputs must not overlap one another or the
 * inputs.  workspace: fp4idx_beam_select_workspace_bytes(n_rows, vocab, k) bytes, 16-byte
 * aligned, nothing in it needs to be initialised; calls that may overlap need one each.
 * Work is shared out over all rows, dead ones too: where one row a group is alive (behind the
 * prompts), the live rows alone with n_beams 1 are faster.
 */
size_t fp4idx_beam_select_workspace_bytes(int64_t max_rows, int32_t vocab, int32_t k);
int fp4idx_beam_select(const void* logits, int32_t logits_type, int64_t logits_stride, int32_t vocab,
                       const float* scores, int64_t n_rows, int32_t n_beams, int32_t k, const int32_t* done,
                       int32_t end_token, void* workspace, size_t workspace_bytes, float* out_scores,
                       int32_t* out_rows, int32_t* out_tokens, int32_t* done_out, int32_t* status_dev, void* stream);

/*
 * Fork of page tables -- the rows of a batch go on as other rows (the beams that were
 * chosen, a prompt that becomes several samples, a batch without its ended sequences),
 * and the pages that no row holds any more go back to the free list of fp4idx_plan_step.
 * Row r of the old table holds ceil(e/64) pages, e = floor(cached_lens[r] / ratio) entries.
 * Row i of the new table goes on from row parents[i] (-1: it is empty):
 *   - it shares all of that row's full pages;
 *   - of the rows that go on from one parent, the first keeps the page that is only partly
 *     filled (unless it is pinned); each other one gets a page of its own, listed in
 *     copy_src / copy_dst: copy these (fp4idx_copy_pages) before the next store.
 * Pages that were held by rows from which none goes on, and by none of the others, and are
 * not pinned, come back, in ascending order.  The first of them serve as the new pages of
 * this call; what is missing is taken from free_pages at *free_head on, what is left over
 * is written just below *free_head.
 *   page_table  [n_old, max_pages] int32, cached_lens [n_old] int32, ratio 1..64
 *   parents     [n_new] int32;  n_old, n_new <= 8192
 *   num_pages   pages of the pool (1..2^23); ids of the table and the list lie below it
 *   pinned      [ceil(num_pages/32)] uint32 bit patterns, nullable: bit p % 32 of word p / 32
 *               is set for a page that something else holds too (a prefix cache); it is
 *               neither freed nor written to
 *   free_pages  [n_free] int32 (read from *free_head on, written below), free_head: device
 *               int32, nullable = 0; n_free may be 0
 *   page_table_out [n_new, max_pages] (written; -1 behind a row's pages), cached_out [n_new]
 *               (written), copy_src, copy_dst [n_new] (written; -1 behind the last copy)
 *   counts [4]  (written): copies, pages that came back, the change of *free_head (new
 *               pages minus pages that came back), rows that go on
 * *free_head is not written: the caller adds counts[2] (a repeated call gives the same
 * result).  A page that is partly filled must be held by no other row (rows that the step
 * plan and this call built are so); such rows may share full pages in any way.
 * The first row whose new page is not in the list, and all behind it that need one, are
 * left empty; if the pages that came back do not fit below *free_head, the lowest of those
 * left over are not listed; if *free_head is outside [0, n_free], none is taken or listed
 * (each CAPACITY; pages lost to the list come back with fp4idx_compact_pages).  A parent
 * outside [-1, n_old) (BAD_PAGE), and one whose length is negative or needs more than
 * max_pages pages (BAD_LENGTH), leave their rows empty; such a parent's pages do not come
 * back.  An id outside [0, num_pages) is handed on as it is and never comes back, a partly
 * filled page with such an id is not copied (BAD_PAGE).  The outputs must not overlap one
 * another or the inputs (page_table_out and cached_out are buffers of their own).
 * A device (or a part of one) that places no cluster of 16 CTAs takes pools of up to 2^22
 * pages, here and in fp4idx_compact_pages; larger ones are a CUDA error there.
 */
int fp4idx_fork_pages(const int32_t* page_table, const int32_t* cached_lens, int64_t n_old, int32_t max_pages,
                      int32_t ratio, const int32_t* parents, int64_t n_new, int64_t num_pages, const uint32_t* pinned,
                      int32_t* free_pages, int64_t n_free, const int32_t* free_head, int32_t* page_table_out,
                      int32_t* cached_out, int32_t* copy_src, int32_t* copy_dst, int32_t* counts, int32_t* status_dev,
                      void* stream);

/*
 * Copies of whole pages, in several caches at once -- the page src[i] of each cache is
 * copied over its page dst[i].
 *   src, dst    [n_copies] int32; a pair with a negative id is padding
 *   count       device int32, nullable: only the first *count pairs are read (counts of
 *               fp4idx_fork_pages and fp4idx_compact_pages)
 *   regions     host array of n_regions (0..256) device pointers, page_bytes host array of the
 *               bytes of a page in each (a multiple of 16, at most 2^30): page p of region c at byte
 *               p*page_bytes[c].  16-byte aligned; read before the call returns.
 *   num_pages   pages in every region (0..2^31-1); a pair with an id from num_pages on is
 *               skipped (BAD_PAGE)
 * No page may be both a source and a destination of one call, or a destination twice
 * (a page copied onto itself stays as it is).
 */
int fp4idx_copy_pages(const int32_t* src, const int32_t* dst, int64_t n_copies, const int32_t* count,
                      void* const* regions, const int64_t* page_bytes, int32_t n_regions, int64_t num_pages,
                      int32_t* status_dev, void* stream);

/*
 * Compaction of a page pool -- the pages in use (held by a row, or pinned) move to the
 * lowest ids, so that the end of the pool can be given away, and the free list is rebuilt
 * from what is in use.  n pages are in use: the i-th page from id n on that is held and not
 * pinned moves to the i-th id below n that is not in use (ascending), for the first
 * max_moves of them.
 *   page_table [n_seqs, max_pages], cached_lens [n_seqs], ratio, num_pages, pinned as
 *              fp4idx_fork_pages; n_seqs <= 65536.  A pinned page keeps its id.
 *   page_table_out [n_seqs, max_pages] (written): the table after the moves, -1 behind a
 *              row's pages
 *   move_src, move_dst [max_moves] int32 (written; -1 behind the last move): copy these
 *              pages (fp4idx_copy_pages) before the next store or read of the cache
 *   free_pages [n_free] int32 (written from index counts[3] on): the ids not in use after
 *              the moves, ascending, at the end of the buffer
 *   counts [4] (written): moves, pages in use, the highest id in use after the moves + 1, the
 *              index of the first free id in free_pages (the new *free_head)
 * Where n_free is less than the ids that are free, the highest n_free of them are listed
 * (CAPACITY).  A row with a negative length or one that needs more than max_pages pages
 * gets an empty table row, and holds nothing (BAD_LENGTH); an id outside [0, num_pages) is
 * handed on as it is (BAD_PAGE).  workspace: fp4idx_compact_pages_workspace_bytes(num_pages)
 * bytes, 16-byte aligned, nothing in it needs to be initialised; calls that may overlap need
 * one each.  The outputs must not overlap one another or the inputs.
 */
size_t fp4idx_compact_pages_workspace_bytes(int64_t num_pages);
int fp4idx_compact_pages(const int32_t* page_table, const int32_t* cached_lens, int64_t n_seqs, int32_t max_pages,
                         int32_t ratio, int64_t num_pages, const uint32_t* pinned, void* workspace,
                         size_t workspace_bytes, int32_t* free_pages, int64_t n_free, int32_t* page_table_out,
                         int32_t* move_src, int32_t* move_dst, int64_t max_moves, int32_t* counts, int32_t* status_dev,
                         void* stream);

/*
 * Test support for the bounded waits of the logits, attention and latent store kernels (failure
 * detection), with no counterpart on the pages.  Every wait of such a pipeline gives up after
 * wait_limit_ns (0 restores the default, 2 s): the CTA then records FP4IDX_ERR_TIMEOUT
 * in status_dev, lets the copies it issued land, frees its tensor memory and returns,
 * and the context stays usable.  idle_producers != 0 tells the producer warps of
 * later launches to issue nothing, so that every launch ends in that timeout;
 * a test sets it with a short limit, checks the status, and calls
 * fp4idx_test_pipeline_waits(0, 0) to restore normal operation.  Process-wide; host
 * only (takes effect at the next launch).
 */
int fp4idx_test_pipeline_waits(int32_t idle_producers, int64_t wait_limit_ns);

/* Copy the device status word to *host_out (host pointer).  Synchronises `stream`:
 * a test/diagnostic helper, not for the hot path. */
int fp4idx_read_status(const int32_t* status_dev, int32_t* host_out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FP4IDX_H */
