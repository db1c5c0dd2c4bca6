// The page pool: page tables forked (shared, copied on write, freed) and compacted.
//
// Both kernels are one cluster of CTAs with one bit a page of the pool in shared memory, the bits
// of adjacent pages dealt out over the CTAs (CTA c holds words [c << shift, (c + 1) << shift)).  Rows of
// the tables are read by all CTAs; a page is marked where its bit lives, through distributed
// shared memory.  Lists in ascending order of ids are then popcounts, one scan a CTA and one
// exchange of the CTAs' sums.  Nothing is left in device memory from call to call.
#include <algorithm>

#include "beam.cuh"
#include "mma_bf16.cuh"

namespace fp4idx {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kMaxCtas = 16;
constexpr int kStep = 128;  // columns that a warp takes at once
constexpr int32_t kNone = INT32_MAX;

struct Cluster {
  int rank, ctas, shift;  // shift: log2 of the words of bits a CTA holds
  uint32_t bits;          // shared-memory address of this CTA's words

  __device__ uint32_t word(int32_t page) const {
    const uint32_t w = (uint32_t)page >> 5;
    return mma::map_shared(bits + ((w & ((1u << shift) - 1)) << 2), w >> shift);
  }
  __device__ void set(int32_t page) const {
    asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(word(page)), "r"(1u << (page & 31)) : "memory");
  }
  __device__ void clear(int32_t page) const {
    asm volatile("red.relaxed.cluster.shared::cluster.and.b32 [%0], %1;" ::"r"(word(page)), "r"(~(1u << (page & 31))) : "memory");
  }
  __device__ bool test(int32_t page) const {
    uint32_t v;
    asm volatile("ld.relaxed.cluster.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(word(page)) : "memory");
    return v >> (page & 31) & 1u;
  }
};

// Sums over the CTA's threads (exclusive, and the total) and over the cluster's CTAs.
struct Scan {
  int32_t warp[kWarps];
  int32_t total;
};
__device__ __forceinline__ int32_t exclusive(int32_t v, Scan& sm, int32_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int32_t s = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int32_t u = __shfl_up_sync(~0u, s, d);
    if (lane >= d) s += u;
  }
  __syncthreads();  // (an earlier scan has been read)
  if (lane == 31) sm.warp[warp] = s;
  __syncthreads();
  if (warp == 0) {
    int32_t w = sm.warp[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int32_t u = __shfl_up_sync(~0u, w, d);
      if (lane >= d) w += u;
    }
    sm.warp[lane] = w;
  }
  __syncthreads();
  *total = sm.warp[kWarps - 1];
  return s - v + (warp ? sm.warp[warp - 1] : 0);
}
// Every CTA's value in all CTAs' tables; read them after the next cluster barrier.
__device__ __forceinline__ void publish(const Cluster& cl, int32_t* table, int32_t v) {
  if ((int)threadIdx.x < cl.ctas)
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mma::map_shared(ptx::smem_addr(table + cl.rank), threadIdx.x)), "r"(v)
                 : "memory");
}
__device__ __forceinline__ int32_t before_me(const Cluster& cl, const int32_t* table, int32_t* total) {
  int32_t mine = 0, all = 0;
  for (int c = 0; c < cl.ctas; c++) {
    if (c == cl.rank) mine = all;
    all += table[c];
  }
  *total = all;
  return mine;
}

// Pages of a row of `len` tokens, -1 if its length is negative or needs more than the table's columns.
__device__ __forceinline__ int32_t pages_of(int32_t len, int32_t ratio, int32_t max_pages) {
  const int32_t n = len / ratio / kPage + (len / ratio % kPage != 0);
  return len < 0 || n > max_pages ? -1 : n;
}

// This thread's share of the CTA's words: `each` words from first on.
struct Share {
  int32_t first, last;
  __device__ Share(const Cluster& cl) {
    const int32_t words = 1 << cl.shift, each = (words + kThreads - 1) / kThreads;
    first = min(words, (int)threadIdx.x * each);
    last = min(words, first + each);
  }
};

// ---------------------------------------------------------------- fork
struct ForkTables {
  Scan scan;
  int32_t freed[kMaxCtas];
};

__global__ void __launch_bounds__(kThreads, 1) fork_kernel(const ForkArgs a, int shift) {
  extern __shared__ __align__(16) uint32_t smem[];
  __shared__ ForkTables sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t* bits = smem;
  int32_t* first = reinterpret_cast<int32_t*>(smem + (1 << shift));  // an old row's first new row
  int32_t* copies = first + a.n_old;                                 // the new rows that get a page
  const Cluster cl{(int)blockIdx.x, (int)gridDim.x, shift, ptx::smem_addr(bits)};
  const bool lead = cl.rank == 0;
  for (int i = tid; i < 1 << shift; i += kThreads) bits[i] = 0;
  for (int i = tid; i < a.n_old; i += kThreads) first[i] = kNone;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __syncthreads();
  for (int i = tid; i < a.n_new; i += kThreads) {
    const int32_t p = a.parents[i];
    if (p >= 0 && p < a.n_old) atomicMin(&first[p], i);
    else if (p != -1 && lead) record_error(a.status, FP4IDX_ERR_BAD_PAGE);
  }
  mma::cluster_sync();

  // the half-filled page of new row i's parent (-1: it has none), and whether i gets one of its own
  auto half_page = [&](int p, int32_t len, int32_t* col) {
    const int32_t e = len / a.ratio;
    *col = e / kPage;
    return e % kPage ? a.page_table[(int64_t)p * a.max_pages + *col] : -1;
  };
  auto own_page = [&](int i, int p, int32_t page) {
    if ((uint32_t)page >= (uint32_t)a.num_pages) return false;
    return first[p] != i || (a.pinned && (a.pinned[page >> 5] >> (page & 31) & 1));
  };
  const int blocks = (a.max_pages + kStep - 1) / kStep, warps = cl.ctas * kWarps, at = cl.rank * kWarps + warp;
  // pages of the rows from which none goes on
  for (int64_t u = at; u < (int64_t)a.n_old * blocks; u += warps) {
    const int r = (int)(u / blocks), c0 = (int)(u - (int64_t)r * blocks) * kStep;
    if (first[r] != kNone) continue;
    const int32_t n = pages_of(a.cached[r], a.ratio, a.max_pages);
    for (int c = c0 + lane; c < min(n, c0 + kStep); c += 32) {
      const int32_t page = a.page_table[(int64_t)r * a.max_pages + c];
      if ((uint32_t)page < (uint32_t)a.num_pages) cl.set(page);
      else record_error(a.status, FP4IDX_ERR_BAD_PAGE);
    }
    if (n < 0 && lane == 0) record_error(a.status, FP4IDX_ERR_BAD_LENGTH);
  }
  // the new rows, but for the pages that this call gives them
  for (int64_t u = at; u < (int64_t)a.n_new * blocks; u += warps) {
    const int i = (int)(u / blocks), c0 = (int)(u - (int64_t)i * blocks) * kStep, p = a.parents[i];
    int32_t n = 0, len = 0, skip = -1;
    if (p >= 0 && p < a.n_old) {
      len = a.cached[p];
      n = pages_of(len, a.ratio, a.max_pages);
      if (n < 0) {
        if (lane == 0) record_error(a.status, FP4IDX_ERR_BAD_LENGTH);
        n = len = 0;
      }
      int32_t col;
      if (n > 0 && own_page(i, p, half_page(p, len, &col))) skip = col;
    }
    for (int c = c0 + lane; c < min(a.max_pages, c0 + kStep); c += 32)
      if (c != skip) a.table_out[(int64_t)i * a.max_pages + c] = c < n ? a.page_table[(int64_t)p * a.max_pages + c] : -1;
    if (c0 == 0 && lane == 0) a.cached_out[i] = len;
  }
  mma::cluster_sync();
  // ... that the other rows hold too
  for (int64_t u = at; u < (int64_t)a.n_old * blocks; u += warps) {
    const int r = (int)(u / blocks), c0 = (int)(u - (int64_t)r * blocks) * kStep;
    if (first[r] == kNone) continue;
    const int32_t n = pages_of(a.cached[r], a.ratio, a.max_pages);
    for (int c = c0 + lane; c < min(n, c0 + kStep); c += 32) {
      const int32_t page = a.page_table[(int64_t)r * a.max_pages + c];
      if ((uint32_t)page >= (uint32_t)a.num_pages) record_error(a.status, FP4IDX_ERR_BAD_PAGE);
      else if (cl.test(page)) cl.clear(page);
    }
  }
  // the rows that get a page, in order (every CTA for itself)
  int32_t n_copies = 0, n_rows = 0;
  for (int base = 0; base < a.n_new; base += kThreads) {
    const int i = base + tid;
    bool goes = false, mine = false;
    if (i < a.n_new) {
      const int32_t p = a.parents[i];
      if (p >= 0 && p < a.n_old) {
        const int32_t len = a.cached[p];
        goes = pages_of(len, a.ratio, a.max_pages) >= 0;
        int32_t col;
        mine = goes && own_page(i, p, half_page(p, len, &col));
      }
    }
    int32_t n;
    const int32_t c = n_copies + exclusive(mine, sm.scan, &n);
    if (mine) copies[c] = i;
    n_copies += n;
    n_rows += __syncthreads_count(goes);
  }
  mma::cluster_sync();
  // the pages that came back
  const Share share(cl);
  const int32_t w0 = cl.rank << shift;
  int32_t mine = 0;
  for (int w = share.first; w < share.last; w++) {
    uint32_t v = bits[w];
    if (v && a.pinned) v &= ~a.pinned[w0 + w];
    bits[w] = v;
    mine += __popc(v);
  }
  int32_t freed_here, n_freed;
  int32_t f = exclusive(mine, sm.scan, &freed_here);
  publish(cl, sm.freed, freed_here);
  mma::cluster_sync();
  f += before_me(cl, sm.freed, &n_freed);
  const int32_t head_in = a.free_head ? *a.free_head : 0;
  const bool good_head = head_in >= 0 && head_in <= a.n_free;
  const int32_t head = good_head ? head_in : 0, avail = good_head ? a.n_free - head : 0;
  const int32_t n_given = (int32_t)min((int64_t)n_copies, (int64_t)n_freed + avail);
  const int32_t left = max(0, n_freed - n_copies), listed = min(left, head), lost = left - listed;
  auto give = [&](int c, int32_t page) {
    const int i = copies[c], p = a.parents[i];
    int32_t col;
    a.copy_src[c] = half_page(p, a.cached[p], &col);
    a.copy_dst[c] = page;
    a.table_out[(int64_t)i * a.max_pages + col] = page;
  };
  for (int w = share.first; w < share.last; w++)
    for (uint32_t v = bits[w]; v; v &= v - 1, f++) {
      const int32_t page = (w0 + w) * 32 + __ffs(v) - 1;
      if (f < n_copies) give(f, page);
      else if (f - n_copies >= lost) a.free_pages[head - listed + (f - n_copies - lost)] = page;
    }
  if (!lead) return;
  for (int c = n_freed + tid; c < n_given; c += kThreads) {
    const int32_t page = a.free_pages[head + (c - n_freed)];
    if ((uint32_t)page >= (uint32_t)a.num_pages) record_error(a.status, FP4IDX_ERR_BAD_PAGE);
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
struct CompactTables {
  Scan scan;
  int32_t used[kMaxCtas], holes[kMaxCtas], movers[kMaxCtas], spare[kMaxCtas], end[kMaxCtas];
};

// Bits of the word that starts at page `p0` for pages in [0, n).
__device__ __forceinline__ uint32_t below(int64_t p0, int32_t n) {
  const int64_t k = n - p0;
  return k >= 32 ? ~0u : k <= 0 ? 0u : (1u << k) - 1u;
}

__global__ void __launch_bounds__(kThreads, 1) compact_kernel(const CompactArgs a, int shift) {
  extern __shared__ __align__(16) uint32_t smem[];
  __shared__ CompactTables sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t* bits = smem;
  const Cluster cl{(int)blockIdx.x, (int)gridDim.x, shift, ptx::smem_addr(bits)};
  const bool lead = cl.rank == 0;
  const int32_t w0 = cl.rank << shift;
  const Share share(cl);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  auto pins = [&](int w) { return a.pinned && (int64_t)(w0 + w) * 32 < a.num_pages ? a.pinned[w0 + w] : 0u; };
  for (int i = tid; i < 1 << shift; i += kThreads) bits[i] = pins(i) & below((int64_t)(w0 + i) * 32, a.num_pages);
  mma::cluster_sync();
  const int blocks = (a.max_pages + kStep - 1) / kStep, warps = cl.ctas * kWarps, at = cl.rank * kWarps + warp;
  for (int64_t u = at; u < (int64_t)a.n_seqs * blocks; u += warps) {
    const int r = (int)(u / blocks), c0 = (int)(u - (int64_t)r * blocks) * kStep;
    const int32_t n = pages_of(a.cached[r], a.ratio, a.max_pages);
    for (int c = c0 + lane; c < min(n, c0 + kStep); c += 32) {
      const int32_t page = a.page_table[(int64_t)r * a.max_pages + c];
      if ((uint32_t)page < (uint32_t)a.num_pages) cl.set(page);
      else record_error(a.status, FP4IDX_ERR_BAD_PAGE);
    }
    if (n < 0 && lane == 0) record_error(a.status, FP4IDX_ERR_BAD_LENGTH);
  }
  mma::cluster_sync();
  int32_t v = 0, here, used;
  for (int w = share.first; w < share.last; w++) v += __popc(bits[w]);
  exclusive(v, sm.scan, &here);
  publish(cl, sm.used, here);
  mma::cluster_sync();
  before_me(cl, sm.used, &used);
  // ids below `used` that are free, and pages from there on that may move
  auto holes = [&](int w) { return ~bits[w] & below((int64_t)(w0 + w) * 32, used); };
  auto movers = [&](int w) { return bits[w] & ~below((int64_t)(w0 + w) * 32, used) & ~pins(w); };
  int32_t nh = 0, nm = 0, here_h, here_m, all_h, all_m;
  for (int w = share.first; w < share.last; w++) nh += __popc(holes(w)), nm += __popc(movers(w));
  int32_t h = exclusive(nh, sm.scan, &here_h);
  int32_t m = exclusive(nm, sm.scan, &here_m);
  publish(cl, sm.holes, here_h);
  publish(cl, sm.movers, here_m);
  mma::cluster_sync();
  h += before_me(cl, sm.holes, &all_h);
  m += before_me(cl, sm.movers, &all_m);
  const int32_t moves = min(all_m, a.max_moves);  // (there are at least as many holes as movers)
  int32_t last = 0, free_here = 0;
  const int32_t m0 = m;
  for (int w = share.first; w < share.last; w++) {
    const int32_t p0 = (w0 + w) * 32;
    uint32_t now = bits[w];
    for (uint32_t x = holes(w); x; x &= x - 1, h++)
      if (h < moves) {
        a.move_dst[h] = p0 + __ffs(x) - 1;
        now |= x & -x;
      }
    for (uint32_t x = movers(w); x; x &= x - 1, m++)
      if (m < moves) {
        a.move_src[m] = p0 + __ffs(x) - 1;
        now &= ~(x & -x);
      }
    bits[w] = now;
    if (now) last = p0 + 32 - __clz(now);
    free_here += __popc(~now & below(p0, a.num_pages));
  }
  int32_t spare, all_spare;
  int32_t f = exclusive(free_here, sm.scan, &spare);
  for (int d = 16; d; d >>= 1) last = max(last, __shfl_xor_sync(~0u, last, d));
  __syncthreads();
  if (lane == 0) sm.scan.warp[warp] = last;
  __syncthreads();
  int32_t end = 0;
  for (int w = 0; w < kWarps; w++) end = max(end, sm.scan.warp[w]);
  publish(cl, sm.spare, spare);
  publish(cl, sm.end, end);
  mma::cluster_sync();
  f += before_me(cl, sm.spare, &all_spare);
  for (int c = 0; c < cl.ctas; c++) end = max(end, sm.end[c]);
  // where the moved pages went
  for (int m1 = m0; m1 < min(m, moves); m1++) a.remap[a.move_src[m1]] = a.move_dst[m1];
  // the free list
  const int32_t listed = min(all_spare, a.n_free), lost = all_spare - listed, head = a.n_free - listed;
  for (int w = share.first; w < share.last; w++)
    for (uint32_t x = ~bits[w] & below((int64_t)(w0 + w) * 32, a.num_pages); x; x &= x - 1, f++)
      if (f >= lost) a.free_pages[head + f - lost] = (w0 + w) * 32 + __ffs(x) - 1;
  mma::cluster_sync();
  for (int64_t u = at; u < (int64_t)a.n_seqs * blocks; u += warps) {
    const int r = (int)(u / blocks), c0 = (int)(u - (int64_t)r * blocks) * kStep;
    const int32_t n = pages_of(a.cached[r], a.ratio, a.max_pages);
    for (int c = c0 + lane; c < min(a.max_pages, c0 + kStep); c += 32) {
      int32_t page = -1;
      if (c < n) {
        page = a.page_table[(int64_t)r * a.max_pages + c];
        if (page >= used && page < a.num_pages && !cl.test(page)) page = a.remap[page];
      }
      a.table_out[(int64_t)r * a.max_pages + c] = page;
    }
  }
  if (lead) {
    for (int c = moves + tid; c < a.max_moves; c += kThreads) a.move_src[c] = a.move_dst[c] = -1;
    if (tid == 0) {
      if (lost > 0) record_error(a.status, FP4IDX_ERR_CAPACITY);
      a.counts[0] = moves;
      a.counts[1] = used;
      a.counts[2] = end;
      a.counts[3] = head;
    }
  }
  mma::cluster_sync();  // no CTA ends while another reads its bits
}

int log2_from(int64_t n) {
  int s = 0;
  while (((int64_t)1 << s) < n) s++;
  return s;
}

// CTAs of a call
int ctas_of(int64_t entries, int64_t pool) { return entries > 16384 || pool > (1 << 18) ? kMaxCtas : 1; }

template <class A>
cudaError_t launch(void (*kernel)(A, int), const A& a, int ctas, int64_t rows, cudaStream_t stream) {
  const int64_t words = ((int64_t)a.num_pages + 31) / 32;
  const int shift = log2_from((words + ctas - 1) / ctas);
  const size_t smem = 4 * (((size_t)1 << shift) + rows);
  const void* f = reinterpret_cast<const void*>(kernel);
  cudaError_t e = set_smem_attr_once(f, 220 * 1024);
  if (e != cudaSuccess) return e;
  if (ctas > 8) {
    int fit = 0;  // (asks for clusters above the portable size)
    e = resident_clusters(f, ctas, kThreads, 220 * 1024, &fit);
    if (e != cudaSuccess) return e;
    if (fit < 1) return cudaErrorInvalidClusterSize;
  }
  return launch_early(kernel, dim3(ctas), kThreads, smem, ctas, stream, a, shift);
}

}  // namespace

cudaError_t launch_fork_pages(const ForkArgs& a, cudaStream_t stream) {
  const int64_t rows = (int64_t)a.n_old + a.n_new;
  return launch(fork_kernel, a, ctas_of(rows * a.max_pages, a.num_pages), rows, stream);
}

cudaError_t launch_compact_pages(const CompactArgs& a, cudaStream_t stream) {
  return launch(compact_kernel, a, ctas_of((int64_t)a.n_seqs * a.max_pages, a.num_pages), 0, stream);
}

}  // namespace fp4idx
