// Beam selection: the k best continuations of each group of rows (beams) over the vocabulary.
//
// total = score + (logit - lse), lse = log sum exp(logit) over the row.  Within a row the order is that
// of the logits, so the scan keeps a row's k largest logits, in lists, next to (largest,
// sum of exp(logit - largest)); the join turns these into lse and totals and picks a group's k best.
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "beam.cuh"

namespace fp4idx {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr float kInf = __builtin_huge_valf();

__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(float v) { return v; }

// What a row contributes: nothing (dead, or its score is no number), its tokens, or its end.
enum Kind : int32_t { kNone, kTokens, kEnd };
__device__ __forceinline__ Kind kind_of(const BeamArgs& a, int row, float score, bool report) {
  if (score == -kInf) return kNone;
  if (!(score < kInf)) {  // NaN or +inf
    if (report) record_error(a.status, FP4IDX_ERR_BAD_VALUE);
    return kNone;
  }
  return a.done && a.done[row] ? kEnd : kTokens;
}

template <class T>
__global__ void __launch_bounds__(kThreads) scan_kernel(const BeamArgs a) {
  __shared__ float sm_v[kWarps], sm_s[kWarps];
  __shared__ int sm_i[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, row = blockIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (kind_of(a, row, a.scores[row], false) != kTokens) return;
  const T* x = static_cast<const T*>(a.logits) + row * a.stride;
  float top = -kInf;
  for (int i = tid; i < a.vocab; i += kThreads) top = fmaxf(top, to_float(x[i]));
  for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
  if (lane == 0) sm_v[warp] = top;
  __syncthreads();
  for (int w = 0; w < kWarps; w++) top = fmaxf(top, sm_v[w]);
  const float ref = top == -kInf ? 0.f : top;
  float sum = 0.f;
  for (int i = tid; i < a.vocab; i += kThreads) sum += expf(to_float(x[i]) - ref);
  for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
  if (lane == 0) sm_s[warp] = sum;
  __syncthreads();
  sum = 0.f;
  for (int w = 0; w < kWarps; w++) sum += sm_s[w];
  // the next one behind (last, at) in descending order, equal ones by their token
  float last = kInf;
  int at = -1, n = 0;
  for (; n < a.k; n++) {
    float v = -kInf;
    int t = a.vocab;
    for (int i = tid; i < a.vocab; i += kThreads) {
      const float u = to_float(x[i]);
      if ((u < last || (u == last && i > at)) && (u > v || (u == v && i < t))) v = u, t = i;
    }
    for (int d = 16; d; d >>= 1) {
      const float u = __shfl_xor_sync(~0u, v, d);
      const int i = __shfl_xor_sync(~0u, t, d);
      if (u > v || (u == v && i < t)) v = u, t = i;
    }
    __syncthreads();
    if (lane == 0) sm_v[warp] = v, sm_i[warp] = t;
    __syncthreads();
    for (int w = 0; w < kWarps; w++)
      if (sm_v[w] > v || (sm_v[w] == v && sm_i[w] < t)) v = sm_v[w], t = sm_i[w];
    if (v == -kInf) break;
    last = v, at = t;
    if (tid == 0) a.lists[(int64_t)row * a.k + n] = BeamItem{v + 0.f, t};
  }
  if (tid == 0) a.stats[row] = BeamStat{top, sum, n, 0};
}

// ---------------------------------------------------------------- join
// A candidate's place: `total` orders first (larger is better), `rest` breaks ties (smaller is better: row,
// then larger logit, then token).  {0, ...}: no candidate.
struct __align__(16) Place {
  uint64_t total, rest;
};
__device__ __forceinline__ bool before(const Place& a, const Place& b) {
  return a.total > b.total || (a.total == b.total && a.rest < b.rest);
}
__device__ __forceinline__ Place place(double total, int beam, float logit, int token) {
  const int64_t t = __double_as_longlong(total + 0.0);
  const int32_t v = __float_as_int(logit);
  const uint32_t up = (uint32_t)v ^ (v < 0 ? 0xFFFFFFFFu : 0x80000000u);
  return Place{(uint64_t)t ^ (t < 0 ? ~0ull : 1ull << 63), (uint64_t)beam << 52 | (uint64_t)~up << 20 | (uint32_t)token};
}

// Descending order; n is a power of two.
__device__ void sort_places(Place* p, int n) {
  for (int size = 2; size <= n; size <<= 1)
    for (int d = size >> 1; d; d >>= 1) {
      __syncthreads();
      for (int i = threadIdx.x; i < n / 2; i += kThreads) {
        const int lo = 2 * i - (i & (d - 1)), hi = lo + d;
        const Place u = p[lo], v = p[hi];
        if (before(v, u) == ((lo & size) == 0)) p[lo] = v, p[hi] = u;
      }
    }
  __syncthreads();
}
__host__ __device__ inline int pow2_from(int n) {
  int p = 1;
  while (p < n) p <<= 1;
  return p;
}

__global__ void __launch_bounds__(kThreads) join_kernel(const BeamArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  Place* pool = reinterpret_cast<Place*>(smem);
  // lse = top + rest, kept apart: next to a large top the sum's logarithm would be lost
  __shared__ float tops[FP4IDX_BEAM_MAX_BEAMS];
  __shared__ double rest[FP4IDX_BEAM_MAX_BEAMS];
  __shared__ float score[FP4IDX_BEAM_MAX_BEAMS];
  __shared__ int32_t kind[FP4IDX_BEAM_MAX_BEAMS];
  __shared__ int32_t open[FP4IDX_BEAM_MAX_K];  // lists that hold a candidate
  __shared__ int32_t n_open, n_found;
  __shared__ Place least;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int first = blockIdx.x * a.beams, k = a.k;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int b = warp; b < a.beams; b += kWarps) {
    const int row = first + b;
    const float s = a.scores[row];
    Kind what = kind_of(a, row, s, lane == 0);
    double total = 0.0;
    float top = -kInf;
    if (what == kTokens) {
      const BeamStat* st = a.stats + (int64_t)row * a.chunks;
      for (int c = lane; c < a.chunks; c += 32) top = fmaxf(top, st[c].top);
      for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
      for (int c = lane; c < a.chunks; c += 32) {
        const float sum = st[c].sum;
        if (sum != 0.f) total += (double)sum * exp(top == -kInf ? 0.0 : (double)st[c].top - top);
      }
      for (int d = 16; d; d >>= 1) total += __shfl_xor_sync(~0u, total, d);
      if (!(total < (double)kInf)) {  // a logit is NaN or +inf
        if (lane == 0) record_error(a.status, FP4IDX_ERR_BAD_VALUE);
        what = kNone;
      } else if (total == 0.0) {
        what = kNone;
      }
      total = log(total);
    }
    if (lane == 0) kind[b] = what, score[b] = s, tops[b] = top, rest[b] = total;
  }
  if (tid == 0) n_open = n_found = 0, least = Place{0, ~0ull};
  __syncthreads();
  // the i-th candidate of list l (list l = beam * chunks + chunk)
  auto size_of = [&](int l) {
    const int b = l / a.chunks, c = l - b * a.chunks;
    return kind[b] == kTokens ? a.stats[(int64_t)(first + b) * a.chunks + c].count : kind[b] == kEnd && c == 0 ? 1 : 0;
  };
  auto item = [&](int l, int i) {
    const int b = l / a.chunks;
    if (kind[b] == kEnd) return place(score[b], b, 0.f, a.end_token);
    const BeamItem it = a.lists[((int64_t)first * a.chunks + l) * k + i];
    return place((double)score[b] + (((double)it.logit - tops[b]) - rest[b]), b, it.logit, it.token);
  };
  // A bound: the k-th best of each list's first `deep` candidates (k candidates at the least, if
  // there are that many).  At most k lists begin with one that is no worse.
  const int lists = a.beams * a.chunks, deep = (k + lists - 1) / lists, heads = pow2_from(lists * deep);
  for (int i = tid; i < heads; i += kThreads) {
    const int l = i / deep, at = i - l * deep;
    pool[i] = l < lists && at < size_of(l) ? item(l, at) : Place{0, ~0ull};
  }
  sort_places(pool, heads);
  if (tid == 0 && k <= heads) least = pool[k - 1];
  __syncthreads();
  for (int l = tid; l < lists; l += kThreads)
    if (size_of(l) > 0 && !before(least, item(l, 0))) open[atomicAdd(&n_open, 1)] = l;
  __syncthreads();
  for (int o = warp; o < n_open; o += kWarps) {
    const int l = open[o], n = size_of(l);
    for (int i = lane; i < n; i += 32) {
      const Place p = item(l, i);
      if (!before(least, p)) pool[atomicAdd(&n_found, 1)] = p;
    }
  }
  __syncthreads();
  const int found = n_found, padded = pow2_from(found);
  for (int i = found + tid; i < padded; i += kThreads) pool[i] = Place{0, ~0ull};
  sort_places(pool, padded);
  for (int i = tid; i < k; i += kThreads) {
    const int64_t o = (int64_t)blockIdx.x * k + i;
    float total = -kInf;
    int row = -1, token = -1, ended = 0;
    if (i < found) {
      const Place p = pool[i];
      const uint64_t t = p.total ^ (p.total >> 63 ? 1ull << 63 : ~0ull);
      total = (float)__longlong_as_double((int64_t)t);
      const int b = (int)(p.rest >> 52);
      row = first + b;
      token = (int)(p.rest & 0xFFFFF);
      ended = kind[b] == kEnd || token == a.end_token;
    }
    a.out_scores[o] = total;
    a.out_rows[o] = row;
    a.out_tokens[o] = token;
    if (a.done_out) a.done_out[o] = ended;
  }
}

int chunks_of(int64_t n_rows, int32_t vocab) { return 1; }

}  // namespace

size_t beam_select_workspace_bytes(int64_t n_rows, int32_t vocab, int32_t k) {
  return (size_t)std::max<int64_t>(1, n_rows) * chunks_of(n_rows, vocab) * (sizeof(BeamStat) + k * sizeof(BeamItem));
}

cudaError_t launch_beam_select(BeamArgs a, int32_t type, void* workspace, cudaStream_t stream) {
  a.chunks = chunks_of(a.n_rows, a.vocab);
  a.stats = static_cast<BeamStat*>(workspace);
  a.lists = reinterpret_cast<BeamItem*>(a.stats + (int64_t)a.n_rows * a.chunks);
  auto scan = type == 0 ? scan_kernel<__nv_bfloat16> : type == 1 ? scan_kernel<__half> : scan_kernel<float>;
  cudaError_t e = launch_early(scan, dim3(a.n_rows), kThreads, 0, 1, stream, a);
  if (e != cudaSuccess) return e;
  const int lists = a.beams * a.chunks, deep = (a.k + lists - 1) / lists;
  const size_t smem = sizeof(Place) * std::max(pow2_from(lists * deep), pow2_from(std::min(lists, a.k) * a.k));
  if (smem > 48 * 1024) {
    e = set_smem_attr_once(reinterpret_cast<const void*>(join_kernel), 64 * 1024);
    if (e != cudaSuccess) return e;
  }
  return launch_early(join_kernel, dim3(a.n_rows / a.beams), kThreads, smem, 1, stream, a);
}

}  // namespace fp4idx
