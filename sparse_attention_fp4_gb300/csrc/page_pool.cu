// The page pool: page tables forked (shared, copied on write, freed) and compacted.
//
// Each kernel is one cluster of CTAs with bits for the pages of the pool in shared memory.  All CTAs read rows of the
// table and mark pages; then CTA c has words [c << shift, (c + 1) << shift) of the marks, and lists of pages in
// ascending order are popcounts, one scan a CTA and one exchange of the CTAs' sums.  Nothing is left in device
// memory from call to call.  Where they fit, every CTA marks a full set of bits of its own, and the
// sets are merged through distributed shared memory (a mark in another CTA's memory costs some four cycles of an
// SM: 130,000 of them took 16 us of a compaction); larger pools are marked where the bits live.
// Both are bound by latency: dependent loads, barriers of the cluster (half a microsecond to one each); large compactions
// by their lists, a word after the other in each warp (14,000 to 19,000 of 43,000 cycles; the two passes over the table
// 12,000, barriers 9,000).  64 rows are forked in 8.9 us (a graph's replay), 256 rows of up to 938 pages in a pool of
// 241,000 in 13.3 us; 64 rows compacted in 12.3 us, 256 in a pool of 245,000 in 22.4 us.
#include <algorithm>

#include "beam.cuh"
#include "mma_bf16.cuh"

namespace fp4idx {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kMaxCtas = 16, kPortable = 8;  // of a cluster: at most, on any device
constexpr int kLane = 8, kStep = 32 * kLane;  // columns that a lane, a warp takes at once
constexpr uint32_t kHalf = 1u << 30;          // beside a row's pages: its last one is partly filled
constexpr size_t kMaxSmem = 225 * 1024;

struct Marks {
  int rank, ctas, shift;
  bool full;     // every CTA has all the words
  uint32_t* own;  // `sets` sets of words

  __device__ int words() const { return full ? ctas << shift : 1 << shift; }
  __device__ int first() const { return full ? rank << shift : 0; }  // of this CTA's share in `own`
  __device__ void set(int32_t page, int set) const {
    uint32_t w = (uint32_t)page >> 5;
    if (full) {
      atomicOr(own + set * words() + w, 1u << (page & 31));
    } else {
      const uint32_t at = set * words() + (w & ((1u << shift) - 1));
      asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(mma::map_shared(ptx::smem_addr(own + at), w >> shift)),
                   "r"(1u << (page & 31))
                   : "memory");
    }
  }
  // Word w of this CTA's share, of all CTAs' marks, in each of `kSets` sets.
  template <int kSets>
  __device__ void merged(int w, uint32_t (&all)[kSets]) const {
    uint32_t v[kSets][kMaxCtas];
#pragma unroll
    for (int s = 0; s < kSets; s++)
#pragma unroll
      for (int c = 0; c < kMaxCtas; c++) {
        const uint32_t* at = own + s * words() + first() + w;
        v[s][c] = c == 0 ? *at : 0;
        if (c > 0 && full && c < ctas)  // (each CTA begins behind itself, so that they do not all read the same one)
          asm volatile("ld.shared::cluster.u32 %0, [%1];"
                       : "=r"(v[s][c])
                       : "r"(mma::map_shared(ptx::smem_addr(at), (rank + c) & (ctas - 1)))
                       : "memory");
      }
#pragma unroll
    for (int s = 0; s < kSets; s++) {
      all[s] = 0;
#pragma unroll
      for (int c = 0; c < kMaxCtas; c++) all[s] |= v[s][c];
    }
  }
};

// The sum of the warps' values before this one, and of all; every lane gives its warp's.
__device__ __forceinline__ int32_t before_warp(int32_t v, int32_t* table, int32_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();  // (an earlier table has been read)
  if (lane == 0) table[warp] = v;
  __syncthreads();
  const int32_t u = table[lane];
  *total = __reduce_add_sync(~0u, u);
  return __reduce_add_sync(~0u, lane < warp ? u : 0);
}
// Every CTA's value in all CTAs' tables; read them after the next cluster barrier.
__device__ __forceinline__ void publish(const Marks& m, int32_t* table, int32_t v) {
  if ((int)threadIdx.x < m.ctas)
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mma::map_shared(ptx::smem_addr(table + m.rank), threadIdx.x)), "r"(v)
                 : "memory");
}
__device__ __forceinline__ int32_t before_cta(const Marks& m, const int32_t* table, int32_t* total) {
  const int lane = threadIdx.x & 31;
  const int32_t u = lane < m.ctas ? table[lane] : 0;
  *total = __reduce_add_sync(~0u, u);
  return __reduce_add_sync(~0u, lane < m.rank ? u : 0);
}

// Pages of a row of `len` tokens, with kHalf where the last is partly filled; -1 if its length is
// negative or needs more than the table's columns.
__device__ __forceinline__ int32_t pages_of(int32_t len, int32_t ratio, int32_t max_pages) {
  const int32_t e = len / ratio, half = e % kPage != 0, n = e / kPage + half;
  return len < 0 || n > max_pages ? -1 : n | (half ? (int32_t)kHalf : 0);
}
__device__ __forceinline__ int32_t count_of(int32_t pages) { return pages < 0 ? 0 : pages & ~kHalf; }

// This warp's words of the CTA's share.
struct Run {
  int32_t first, last;
  __device__ explicit Run(const Marks& m) {
    const int32_t words = 1 << m.shift, each = (words + kWarps - 1) / kWarps, warp = threadIdx.x >> 5;
    first = min(words, warp * each);
    last = min(words, first + each);
  }
};
// Bits of the word that starts at page `p0` for pages in [0, n).
__device__ __forceinline__ uint32_t below(int32_t p0, int32_t n) {
  const int32_t k = n - p0;
  return k >= 32 ? ~0u : k <= 0 ? 0u : (1u << k) - 1u;
}

// f(row, first column, of(row)) for the blocks of kStep columns of a table, a warp each; of(row) is called a block ahead.
// `back`: the warps in reverse order, so that two short tables are read by different warps.
template <class Of, class F>
__device__ __forceinline__ void each_block(const Marks& m, bool back, int32_t rows, int32_t max_pages, Of&& of, F&& f) {
  const uint32_t blocks = (max_pages + kStep - 1) / kStep, all = rows * blocks, step = m.ctas * kWarps;
  const uint32_t at = m.rank * kWarps + (threadIdx.x >> 5);
  uint32_t u = back ? step - 1 - at : at;
  if (u >= all) return;
  uint32_t r = u / blocks;
  int32_t value = of((int)r);
  while (true) {
    const uint32_t c0 = (u - r * blocks) * kStep, here = r;
    const int32_t now = value;
    const bool more = all - u > step;
    if (more) {
      u += step;
      r = u / blocks;
      value = of((int)r);
    }
    f((int)here, (int)c0, now);
    if (!more) return;
  }
}
// A lane's entries of a block of a row with n pages, -1 behind them.
__device__ __forceinline__ void load_block(const int32_t* row, int c0, int32_t n, int32_t (&page)[kLane]) {
#pragma unroll
  for (int j = 0; j < kLane; j++) {
    const int c = c0 + j * 32 + (threadIdx.x & 31);
    page[j] = c < n ? row[c] : -1;
  }
}
// Marks a row's block; ids outside the pool are reported.
__device__ __forceinline__ void mark_block(const Marks& m, const int32_t* row, int c0, int32_t n, int set, int32_t num_pages,
                                           int32_t* status) {
  if (c0 >= n) return;
  int32_t page[kLane];
  load_block(row, c0, n, page);
#pragma unroll
  for (int j = 0; j < kLane; j++) {
    if ((uint32_t)page[j] < (uint32_t)num_pages) m.set(page[j], set);
    else if (c0 + j * 32 + (int)(threadIdx.x & 31) < n) record_error(status, FP4IDX_ERR_BAD_PAGE);
  }
}

// ---------------------------------------------------------------- fork
constexpr int32_t kNoRow = INT32_MAX;

__global__ void __launch_bounds__(kThreads, 1) fork_kernel(const ForkArgs a, int shift, bool full) {
  extern __shared__ __align__(16) uint32_t smem[];
  __shared__ int32_t table[kWarps], freed[kMaxCtas];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Marks m{(int)blockIdx.x, (int)gridDim.x, shift, full, smem};
  constexpr int kGone = 0, kStays = 1;  // pages of rows from which none, or one at the least goes on
  const int words = m.words();
  int32_t* first = reinterpret_cast<int32_t*>(smem + 2 * words);  // an old row's first new row
  int32_t* pages = first + a.n_old;
  int16_t* parent = reinterpret_cast<int16_t*>(pages + a.n_old);
  int16_t* copies = parent + a.n_new;  // the new rows that get a page of their own
  const bool lead = m.rank == 0;
  for (int i = tid; i < 2 * words; i += kThreads) smem[i] = 0;
  for (int i = tid; i < a.n_old; i += kThreads) first[i] = kNoRow;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int32_t head_in = a.free_head ? *a.free_head : 0;
  __syncthreads();
  for (int i = tid; i < max(a.n_old, a.n_new); i += kThreads) {
    const int32_t len = i < a.n_old ? a.cached[i] : 0, p = i < a.n_new ? a.parents[i] : -1;
    if (i < a.n_old) {
      pages[i] = pages_of(len, a.ratio, a.max_pages);
      if (pages[i] < 0 && lead) record_error(a.status, FP4IDX_ERR_BAD_LENGTH);
    }
    if (i < a.n_new) {
      const bool good = p >= 0 && p < a.n_old;
      if (good) atomicMin(&first[p], i);
      else if (p != -1 && lead) record_error(a.status, FP4IDX_ERR_BAD_PAGE);
      parent[i] = good ? (int16_t)p : (int16_t)-1;
    }
  }
  if (full) __syncthreads();
  else mma::cluster_sync();  // (all CTAs' words are clear)

  // whether new row i gets a page of its own for the partly filled `page` of its parent
  auto own_page = [&](int i, int p, int32_t page) {
    if ((uint32_t)page >= (uint32_t)a.num_pages) return false;
    return first[p] != i || (a.pinned && (a.pinned[page >> 5] >> (page & 31) & 1));
  };
  each_block(m, false, a.n_old, a.max_pages, [&](int r) { return pages[r]; }, [&](int r, int c0, int32_t has) {
    mark_block(m, a.page_table + (int64_t)r * a.max_pages, c0, count_of(has), first[r] == kNoRow ? kGone : kStays, a.num_pages,
               a.status);
  });
  // the new rows, but for the pages that this call gives them
  each_block(m, true, a.n_new, a.max_pages, [&](int i) { return (int32_t)parent[i]; }, [&](int i, int c0, int32_t p) {
    const int32_t has = p < 0 ? 0 : pages[p], n = count_of(has);
    int32_t page[kLane];
    load_block(a.page_table + (int64_t)p * a.max_pages, c0, n, page);
#pragma unroll
    for (int j = 0; j < kLane; j++) {
      const int c = c0 + j * 32 + lane;
      const bool given = has > 0 && (has & kHalf) && c == n - 1 && own_page(i, p, page[j]);
      if (c < a.max_pages && !given) a.table_out[(int64_t)i * a.max_pages + c] = page[j];
    }
    if (c0 == 0 && lane == 0) a.cached_out[i] = has < 0 || p < 0 ? 0 : a.cached[p];
  });
  // the rows that get a page, in order (every CTA for itself)
  int32_t n_copies = 0, n_rows = 0;
  for (int base = 0; base < a.n_new; base += kThreads) {
    const int i = base + tid;
    const int p = i < a.n_new ? parent[i] : -1;
    const int32_t has = p < 0 ? -1 : pages[p];
    const bool mine = has > 0 && (has & kHalf) && own_page(i, p, a.page_table[(int64_t)p * a.max_pages + count_of(has) - 1]);
    const uint32_t set = __ballot_sync(~0u, mine);
    int32_t n;
    const int32_t c = n_copies + before_warp(__popc(set), table, &n) + __popc(set & ((1u << lane) - 1));
    if (mine) copies[c] = (int16_t)i;
    n_copies += n;
    n_rows += __syncthreads_count(has >= 0);
  }
  mma::cluster_sync();
  // the pages that come back: this CTA's share, in place of its marks
  const Run run(m);
  const int32_t w0 = m.rank << shift;
  uint32_t* back = smem + m.first();
  for (int w = tid; w < 1 << shift; w += kThreads) {
    const uint32_t pin = a.pinned && w0 + w < (a.num_pages + 31) / 32 ? a.pinned[w0 + w] : 0u;
    uint32_t held[2];
    m.merged(w, held);
    back[w] = held[kGone] & ~held[kStays] & ~pin;
  }
  __syncthreads();
  int32_t mine = 0;
  for (int w = run.first + lane; w < run.last; w += 32) mine += __popc(back[w]);
  int32_t freed_here, n_freed;
  int32_t f = before_warp(__reduce_add_sync(~0u, mine), table, &freed_here);
  publish(m, freed, freed_here);
  mma::cluster_sync();
  f += before_cta(m, freed, &n_freed);
  const bool good_head = head_in >= 0 && head_in <= a.n_free;
  const int32_t head = good_head ? head_in : 0, avail = good_head ? a.n_free - head : 0;
  const int32_t n_given = (int32_t)min((int64_t)n_copies, (int64_t)n_freed + avail);
  const int32_t left = max(0, n_freed - n_copies), listed = min(left, head), lost = left - listed;
  auto give = [&](int c, int32_t page) {  // copy_dst[c] is written
    const int i = copies[c], p = parent[i];
    const int64_t col = count_of(pages[p]) - 1;
    a.copy_src[c] = a.page_table[(int64_t)p * a.max_pages + col];
    a.table_out[(int64_t)i * a.max_pages + col] = page;
  };
  int32_t unused;
  const int32_t first_here = before_cta(m, freed, &unused);
  for (int w = run.first; w < run.last; w++) {
    const uint32_t v = back[w];
    if (v == 0) continue;
    if (v >> lane & 1) {
      const int32_t at = f + __popc(v & ((1u << lane) - 1)), page = (w0 + w) * 32 + lane;
      if (at < n_copies) a.copy_dst[at] = page;
      else if (at - n_copies >= lost) a.free_pages[head - listed + (at - n_copies - lost)] = page;
    }
    f += __popc(v);
  }
  __syncthreads();
  for (int c = first_here + tid; c < min(first_here + freed_here, n_copies); c += kThreads) give(c, a.copy_dst[c]);
  if (!lead) return;
  for (int c = n_freed + tid; c < n_given; c += kThreads) {
    const int32_t page = a.free_pages[head + (c - n_freed)];
    if ((uint32_t)page >= (uint32_t)a.num_pages) record_error(a.status, FP4IDX_ERR_BAD_PAGE);
    a.copy_dst[c] = page;
    give(c, page);
  }
  for (int c = n_given + warp; c < n_copies; c += kWarps) {
    const int i = copies[c];
    for (int col = lane; col < a.max_pages; col += 32) a.table_out[(int64_t)i * a.max_pages + col] = -1;
    if (lane == 0) a.cached_out[i] = 0;
  }
  for (int c = n_given + tid; c < a.n_new; c += kThreads) a.copy_src[c] = a.copy_dst[c] = -1;
  if (tid == 0) {
    if (!good_head || n_given < n_copies || lost > 0) record_error(a.status, FP4IDX_ERR_CAPACITY);
    a.counts[0] = n_given;
    a.counts[1] = n_freed;
    a.counts[2] = n_freed > n_copies ? -listed : n_given - n_freed;
    a.counts[3] = n_rows - (n_copies - n_given);
  }
}

// ---------------------------------------------------------------- compaction
__global__ void __launch_bounds__(kThreads, 1) compact_kernel(const CompactArgs a, int shift, bool full) {
  extern __shared__ __align__(16) uint32_t smem[];
  __shared__ int32_t table[kWarps], used_by[kMaxCtas], holes_by[kMaxCtas], movers_by[kMaxCtas], spare_by[kMaxCtas], end_by[kMaxCtas];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Marks m{(int)blockIdx.x, (int)gridDim.x, shift, full, smem};
  const bool lead = m.rank == 0;
  for (int i = tid; i < m.words(); i += kThreads) smem[i] = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (full) __syncthreads();
  else mma::cluster_sync();
  auto len_of = [&](int r) { return a.cached[r]; };
  each_block(m, false, a.n_seqs, a.max_pages, len_of, [&](int r, int c0, int32_t len) {
    const int32_t n = pages_of(len, a.ratio, a.max_pages);
    if (n < 0 && lane == 0) record_error(a.status, FP4IDX_ERR_BAD_LENGTH);
    mark_block(m, a.page_table + (int64_t)r * a.max_pages, c0, count_of(n), 0, a.num_pages, a.status);
  });
  mma::cluster_sync();
  // this CTA's share of the pages in use, in place of its marks, and of those that may move
  const Run run(m);
  const int32_t w0 = m.rank << shift;
  uint32_t *bits = smem + m.first(), *free_to_move = smem + m.words();
  auto page0 = [&](int w) { return (w0 + w) * 32; };
  auto pins = [&](int w) { return a.pinned && page0(w) < a.num_pages ? a.pinned[w0 + w] & below(page0(w), a.num_pages) : 0u; };
  for (int w = tid; w < 1 << shift; w += kThreads) {
    const uint32_t pin = pins(w);
    uint32_t held[1];
    m.merged(w, held);
    bits[w] = held[0] | pin;
    free_to_move[w] = held[0] & ~pin;
  }
  __syncthreads();
  int32_t n = 0, here, used;
  for (int w = run.first + lane; w < run.last; w += 32) n += __popc(bits[w]);
  before_warp(__reduce_add_sync(~0u, n), table, &here);
  publish(m, used_by, here);
  mma::cluster_sync();
  before_cta(m, used_by, &used);
  // ids below `used` that are free, and pages from there on that may move
  auto holes = [&](int w) { return ~bits[w] & below(page0(w), used); };
  auto movers = [&](int w) { return free_to_move[w] & ~below(page0(w), used); };
  int32_t nh = 0, nm = 0, here_h, here_m, all_m, unused;
  for (int w = run.first + lane; w < run.last; w += 32) nh += __popc(holes(w)), nm += __popc(movers(w));
  int32_t h = before_warp(__reduce_add_sync(~0u, nh), table, &here_h);
  int32_t v = before_warp(__reduce_add_sync(~0u, nm), table, &here_m);
  publish(m, holes_by, here_h);
  publish(m, movers_by, here_m);
  mma::cluster_sync();
  h += before_cta(m, holes_by, &unused);
  v += before_cta(m, movers_by, &all_m);
  const int32_t moves = min(all_m, a.max_moves);  // (there are at least as many holes as movers)
  const int32_t first_mover = v;
  const uint32_t before = (1u << lane) - 1;
  for (int w = run.first; w < run.last && h < moves; w++) {
    const int32_t p0 = page0(w);
    if (p0 >= used) break;
    const uint32_t open = holes(w);
    if (open == 0) continue;
    const int32_t at = h + __popc(open & before);
    const bool fills = (open >> lane & 1) && at < moves;
    if (fills) a.move_dst[at] = p0 + lane;
    h += __popc(open);
    const uint32_t filled = __ballot_sync(~0u, fills);
    if (lane == 0) bits[w] |= filled;
  }
  for (int w = run.first; w < run.last && v < moves; w++) {
    const int32_t p0 = page0(w);
    const uint32_t from = movers(w);
    if (from == 0) continue;
    const int32_t at = v + __popc(from & before);
    const bool goes = (from >> lane & 1) && at < moves;
    if (goes) a.move_src[at] = p0 + lane;
    v += __popc(from);
    const uint32_t gone = __ballot_sync(~0u, goes);
    if (lane == 0) bits[w] &= ~gone;
  }
  __syncwarp();
  int32_t last = 0, spare = 0;
  for (int w = run.first + lane; w < run.last; w += 32) {
    if (bits[w]) last = page0(w) + 32 - __clz(bits[w]);
    spare += __popc(~bits[w] & below(page0(w), a.num_pages));
  }
  spare = __reduce_add_sync(~0u, spare);
  last = (int32_t)__reduce_max_sync(~0u, (uint32_t)last);
  int32_t here_spare, all_spare;
  int32_t f = before_warp(spare, table, &here_spare);
  publish(m, spare_by, here_spare);
  __syncthreads();
  if (lane == 0) table[warp] = last;
  __syncthreads();
  publish(m, end_by, (int32_t)__reduce_max_sync(~0u, (uint32_t)table[lane]));
  mma::cluster_sync();
  f += before_cta(m, spare_by, &all_spare);
  const int32_t end = (int32_t)__reduce_max_sync(~0u, lane < m.ctas ? (uint32_t)end_by[lane] : 0u);
  // where the pages from `used` on are now: those of this CTA's share that move, and those that stay
  for (int i = first_mover + lane; i < min(v, moves); i += 32) a.remap[a.move_src[i]] = a.move_dst[i];
  const int32_t listed = min(all_spare, a.n_free), lost = all_spare - listed, head = a.n_free - listed;
  int32_t* free_at = a.free_pages + (head - lost);
  for (int w = run.first; w < run.last; w++) {
    const int32_t p0 = page0(w);
    const uint32_t now = bits[w], open = ~now & below(p0, a.num_pages);
    if (now && p0 + 32 > used && (now & ~below(p0, used)) >> lane & 1) a.remap[p0 + lane] = p0 + lane;
    if (open == 0) continue;
    const int32_t at = f + (open == ~0u ? lane : __popc(open & before));
    if ((open >> lane & 1) && at >= lost) free_at[at] = p0 + lane;
    f += open == ~0u ? 32 : __popc(open);
  }
  mma::cluster_sync();
  each_block(m, false, a.n_seqs, a.max_pages, len_of, [&](int r, int c0, int32_t len) {
    int32_t page[kLane];
    load_block(a.page_table + (int64_t)r * a.max_pages, c0, count_of(pages_of(len, a.ratio, a.max_pages)), page);
#pragma unroll
    for (int j = 0; j < kLane; j++)
      if (page[j] >= used && page[j] < a.num_pages) page[j] = a.remap[page[j]];
#pragma unroll
    for (int j = 0; j < kLane; j++) {
      const int c = c0 + j * 32 + lane;
      if (c < a.max_pages) a.table_out[(int64_t)r * a.max_pages + c] = page[j];
    }
  });
  if (!lead) return;
  // (counted without a sign: the last step of a list of nearly 2^31 moves passes it)
  for (uint32_t c = moves + tid; c < (uint32_t)a.max_moves; c += kThreads) a.move_src[c] = a.move_dst[c] = -1;
  if (tid == 0) {
    if (lost > 0) record_error(a.status, FP4IDX_ERR_CAPACITY);
    a.counts[0] = moves;
    a.counts[1] = used;
    a.counts[2] = end;
    a.counts[3] = head;
  }
}

int log2_from(int64_t n) {
  int s = 0;
  while (((int64_t)1 << s) < n) s++;
  return s;
}

// CTAs of a call: one for every so many entries of its tables (60 rows forked into 360 12.0 us with 2,048, 14.3 with
// 16,384, 18.4 with 32,768; a compaction of 245,000 pages 31 with up to 16,384, 49 with 32,768, then)
constexpr int64_t kEntries = 2048;

int ctas_of(int64_t entries, int64_t pool) {
  if (pool > (1 << 19)) return kMaxCtas;
  int c = 1;
  while (c < kMaxCtas && c * kEntries < entries) c *= 2;
  return c;
}

template <class A>
cudaError_t launch(void (*kernel)(A, int, bool), const A& a, int sets, int share, int64_t entries, size_t rows,
                   cudaStream_t stream) {
  const int64_t words = ((int64_t)a.num_pages + 31) / 32;
  const void* f = reinterpret_cast<const void*>(kernel);
  cudaError_t e = set_smem_attr_once(f, kMaxSmem);
  if (e != cudaSuccess) return e;
  int ctas = ctas_of(entries, a.num_pages);
  if (ctas > kPortable) {
    int fit = 0;  // (asks for clusters above the portable size, of any call's memory)
    e = resident_clusters(f, ctas, kThreads, kMaxSmem, &fit);
    if (e != cudaSuccess) return e;
    if (fit < 1) ctas = kPortable;
  }
  const int shift = log2_from((words + ctas - 1) / ctas);
  const size_t part = 4 * ((size_t)sets << shift);
  rows += share * ((size_t)4 << shift);
  const bool full = part * ctas + rows <= kMaxSmem;
  const size_t smem = (full ? part * ctas : part) + rows;
  // (sixteen CTAs hold the marks of every pool, eight those of up to 2^22 pages; 256 long rows are forked in 13.1 us by
  // sixteen, 17.8 by eight, a pool of 245,000 pages compacted in 22.4 and 34.5)
  if (smem > kMaxSmem) return cudaErrorInvalidClusterSize;
  return launch_early(kernel, dim3(ctas), kThreads, smem, ctas, stream, a, shift, full);
}

}  // namespace

cudaError_t launch_fork_pages(const ForkArgs& a, cudaStream_t stream) {
  return launch(fork_kernel, a, 2, 0, ((int64_t)a.n_old + a.n_new) * a.max_pages, 8 * (size_t)a.n_old + 4 * (size_t)a.n_new, stream);
}

cudaError_t launch_compact_pages(const CompactArgs& a, cudaStream_t stream) {
  return launch(compact_kernel, a, 1, 1, (int64_t)a.n_seqs * a.max_pages, 0, stream);
}

}  // namespace fp4idx
