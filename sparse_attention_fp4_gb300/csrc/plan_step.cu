// Step plan: page table, slots, positions, sequences and context lengths of a step's rows,
// from request lengths.
//
// One 1,024-thread CTA, or one for every two thousand rows and entries (65,536 rows: 18 us on
// eight CTAs, 11 us on 64).  Few rows are bound by the latency of the chain, many by instructions
// (a search and a division a row; 55 % of the issue slots at 65,536 rows), none by the 1.3 MB.
// Every CTA scans all the sequences itself, 1,024 at a time (four running sums: rows, stored
// entries, pages, entries after the step), which costs less than handing the sums from one
// CTA to another; the rows, entries and pages of each 1,024 sequences are then dealt out over
// all the threads, each finding its sequence by a binary search of the chunk's sums in shared
// memory.  The sums are non-decreasing, so the sequences that fit form a prefix.  No CTA reads
// what another writes: the table entries read are those of pages that exist already.
#include <algorithm>

#include "latent.cuh"

namespace fp4idx {
namespace {

constexpr int kThreads = 1024;
constexpr int32_t kMaxPageId = (1 << 25) - 1;  // slots are int32

// Rows, stored entries, pages, entries after the step.
struct Sums {
  int64_t x, y, z, w;
  Sums() = default;
  __device__ Sums(int64_t x_, int64_t y_, int64_t z_, int64_t w_) : x(x_), y(y_), z(z_), w(w_) {}
};

struct Chunk {
  // inclusive sums within the chunk, for its planned sequences
  int32_t rows[kThreads], stores[kThreads], pages[kThreads];
  int32_t cached[kThreads], entries0[kThreads], pages0[kThreads];
  Sums warp[kThreads / 32];
  Sums total;  // sums of the planned sequences of the chunk
};

__device__ __forceinline__ Sums add4(const Sums& a, const Sums& b) {
  return Sums(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}
__device__ __forceinline__ Sums up4(const Sums& a, int d) {
  return Sums(__shfl_up_sync(~0u, a.x, d), __shfl_up_sync(~0u, a.y, d), __shfl_up_sync(~0u, a.z, d),
                        __shfl_up_sync(~0u, a.w, d));
}
__device__ __forceinline__ Sums warp_scan(Sums v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const Sums u = up4(v, d);
    if (lane >= d) v = add4(v, u);
  }
  return v;
}
// Smallest i in [0, n) whose inclusive sum exceeds v; v < sums[n - 1].
__device__ __forceinline__ int find(const int32_t* sums, int n, int32_t v) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] > v) hi = mid; else lo = mid + 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads, 1) plan_step_kernel(const PlanArgs a) {
  __shared__ Chunk sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int at = blockIdx.x * kThreads + tid, step = gridDim.x * kThreads;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const bool first = blockIdx.x == 0;
  int64_t head = a.free_head ? *a.free_head : 0;
  int64_t avail = (int64_t)a.n_free - head;
  if (head < 0 || avail < 0) {
    if (at == 0) record_error(a.status, FP4IDX_ERR_CAPACITY);
    avail = 0;
    head = 0;
  }
  Sums carry = Sums(0, 0, 0, 0);  // of the planned sequences before this chunk
  int planned = 0;
  bool full = false;
  if (first && tid == 0) {
    a.cu_rows[0] = 0;
    a.cu_context[0] = 0;
  }
  for (int base = 0; base < a.n_seqs; base += kThreads) {
    const int b = base + tid;
    Sums v = Sums(0, 0, 0, 0);
    int32_t c = 0;
    int64_t e0 = 0, p0 = 0;
    if (b < a.n_seqs && !full) {
      c = a.cached[b];
      const int32_t n = a.fresh[b];
      const int64_t end = (int64_t)c + n, e1 = end / a.ratio;
      if (c < 0 || n < 0 || end > INT32_MAX || e1 > (int64_t)a.max_pages * kPage) {
        if (first) record_error(a.status, FP4IDX_ERR_BAD_LENGTH);
      } else {
        e0 = c / a.ratio;
        p0 = (e0 + kPage - 1) / kPage;
        v = Sums(n, e1 - e0, (e1 + kPage - 1) / kPage - p0, e1);
      }
    }
    Sums incl = warp_scan(v, lane);
    __syncthreads();  // the chunk before has been dealt out
    if (lane == 31) sm.warp[warp] = incl;
    __syncthreads();
    if (warp == 0) sm.warp[lane] = warp_scan(sm.warp[lane], lane);
    __syncthreads();
    if (warp > 0) incl = add4(incl, sm.warp[warp - 1]);
    const Sums sum = add4(carry, incl);
    const bool fits = b < a.n_seqs && !full && sum.x <= a.max_rows && sum.y <= a.max_stores && sum.z <= avail &&
                      sum.w <= INT32_MAX;
    const int n_fit = __syncthreads_count(fits);  // a prefix of the chunk
    if (fits) {
      sm.rows[tid] = (int32_t)incl.x;
      sm.stores[tid] = (int32_t)incl.y;
      sm.pages[tid] = (int32_t)incl.z;
      sm.cached[tid] = c;
      sm.entries0[tid] = (int32_t)e0;
      sm.pages0[tid] = (int32_t)p0;
      if (tid == n_fit - 1) sm.total = incl;
    }
    if (n_fit == 0 && tid == 0) sm.total = Sums(0, 0, 0, 0);
    __syncthreads();
    const Sums total = sm.total;
    if (first && b < a.n_seqs) {
      a.cu_rows[b + 1] = (int32_t)(fits ? sum.x : carry.x + total.x);
      a.cu_context[b + 1] = (int32_t)(fits ? sum.w : carry.w + total.w);
    }
    for (int i = at; i < total.x; i += step) {
      const int s = find(sm.rows, n_fit, i);
      const int32_t p = sm.cached[s] + i - (s ? sm.rows[s - 1] : 0);
      const int64_t o = carry.x + i;
      a.q_positions[o] = p;
      a.row_seq[o] = base + s;
      a.context_lens[o] = (int32_t)(((int64_t)p + 1) / a.ratio);
    }
    for (int i = at; i < total.z; i += step) {
      const int s = find(sm.pages, n_fit, i);
      const int32_t col = sm.pages0[s] + i - (s ? sm.pages[s - 1] : 0);
      a.page_table[(int64_t)(base + s) * a.max_pages + col] = a.free_pages[head + carry.z + i];
    }
    for (int i = at; i < total.y; i += step) {
      const int s = find(sm.stores, n_fit, i);
      const int32_t e = sm.entries0[s] + i - (s ? sm.stores[s - 1] : 0);
      const int32_t col = e / kPage, fresh = col - sm.pages0[s];
      // a page taken in this call comes from the list itself: its table entry may be
      // another thread's to write
      const int32_t page = fresh >= 0 ? a.free_pages[head + carry.z + (s ? sm.pages[s - 1] : 0) + fresh]
                                      : a.page_table[(int64_t)(base + s) * a.max_pages + col];
      const bool good = page >= 0 && page <= kMaxPageId;
      if (!good) record_error(a.status, FP4IDX_ERR_BAD_PAGE);
      const int64_t o = carry.y + i;
      a.store_positions[o] = e;
      a.store_slots[o] = good ? page * kPage + e % kPage : -1;
    }
    carry = add4(carry, total);
    planned += n_fit;
    full = full || n_fit < min(kThreads, a.n_seqs - base);
  }
  if (full && at == 0) record_error(a.status, FP4IDX_ERR_CAPACITY);
  for (int64_t i = carry.x + at; i < a.max_rows; i += step) {
    a.q_positions[i] = 0;
    a.row_seq[i] = 0;
    a.context_lens[i] = 0;
  }
  for (int64_t i = carry.y + at; i < a.max_stores; i += step) {
    a.store_positions[i] = 0;
    a.store_slots[i] = -1;
  }
  if (at == 0) {
    a.counts[0] = (int32_t)carry.x;
    a.counts[1] = (int32_t)carry.y;
    a.counts[2] = (int32_t)carry.z;
    a.counts[3] = planned;
  }
}

}  // namespace

cudaError_t launch_plan_step(const PlanArgs& a, cudaStream_t stream) {
  int sms = 0, dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int64_t items = (int64_t)a.max_rows + a.max_stores;
  const int ctas = (int)std::max<int64_t>(1, std::min<int64_t>(sms, items / (2 * kThreads)));
  return launch_early(plan_step_kernel, dim3(ctas), kThreads, 0, 1, stream, a);
}

}  // namespace fp4idx
