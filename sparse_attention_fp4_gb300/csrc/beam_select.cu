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

// ---------------------------------------------------------------- scan
constexpr int kSlots = 128;        // threads of a chunk that may hold candidates
constexpr int kFound = kThreads;   // candidates of a chunk before the last ranking
constexpr int kSegments = 128;

template <class T>
struct Elems;  // sixteen bytes of logits
template <>
struct Elems<__nv_bfloat16> {
  static constexpr uint32_t kMasked = 0xFF80FF80u;  // -inf
  using Pair = __nv_bfloat162;
  __device__ static float2 pair(uint32_t w) { return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); }
};
template <>
struct Elems<__half> {
  static constexpr uint32_t kMasked = 0xFC00FC00u;
  using Pair = __half2;
  __device__ static float2 pair(uint32_t w) { return __half22float2(*reinterpret_cast<__half2*>(&w)); }
};
template <>
struct Elems<float> {
  static constexpr uint32_t kMasked = 0xFF800000u;
};
__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
// f(e, value) for the elements of a vector
template <class T, class F>
__device__ __forceinline__ void each(const uint4& v, F&& f) {
#pragma unroll
  for (int i = 0; i < 4; i++) {
    if constexpr (sizeof(T) == 4) {
      f(i, __uint_as_float(word_of(v, i)));
    } else {
      const float2 p = Elems<T>::pair(word_of(v, i));
      f(2 * i, p.x);
      f(2 * i + 1, p.y);
    }
  }
}
// The largest element (NaN left out).
template <class T, int kVecs>
__device__ __forceinline__ float largest(const uint4 (&v)[kVecs]) {
  if constexpr (sizeof(T) == 4) {
    float m = -kInf;
#pragma unroll
    for (int j = 0; j < kVecs; j++)
      m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(v[j].x), __uint_as_float(v[j].y)),
                         fmaxf(__uint_as_float(v[j].z), __uint_as_float(v[j].w))));
    return m;
  } else {
    using P = typename Elems<T>::Pair;
    uint32_t w = Elems<T>::kMasked;
    P m = *reinterpret_cast<P*>(&w);
#pragma unroll
    for (int j = 0; j < kVecs; j++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        uint32_t u = word_of(v[j], i);
        m = __hmax2(m, *reinterpret_cast<P*>(&u));
      }
    const float2 f = Elems<T>::pair(*reinterpret_cast<uint32_t*>(&m));
    return fmaxf(f.x, f.y);
  }
}
__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint4 load_once(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
// A vector that reaches over the row's first or last token: nothing outside is read.
template <class T>
__device__ __noinline__ uint4 load_edge(const T* x, int p0, int vocab) {
  constexpr int kE = 16 / sizeof(T);
  uint4 v = make_uint4(Elems<T>::kMasked, Elems<T>::kMasked, Elems<T>::kMasked, Elems<T>::kMasked);
  T* e = reinterpret_cast<T*>(&v);
  for (int i = 0; i < kE; i++)
    if (p0 + i >= 0 && p0 + i < vocab) e[i] = x[p0 + i];
  return v;
}
// Numbers in the order of their bits; larger is larger.
__device__ __forceinline__ uint32_t ordered(float v) {
  const int32_t i = __float_as_int(v + 0.f);
  return (uint32_t)i ^ (i < 0 ? 0xFFFFFFFFu : 0x80000000u);
}

template <int kVecs>
struct ScanShared {
  uint4 slot[kSlots][kVecs];
  float segment[kSegments];
  float top[kWarps], sum[kWarps];
  BeamItem found[kFound];
  int32_t owner[kSlots];
  int32_t slots, n, count[2];
  float bound;
};

// A sum over the CTA; `slot` alternates from call to call.
__device__ __forceinline__ int block_sum(int v, int32_t* count, int slot) {
  v = __reduce_add_sync(~0u, v);
  if ((threadIdx.x & 31) == 0) atomicAdd(&count[slot], v);
  __syncthreads();
  const int all = count[slot];
  if (threadIdx.x == 0) count[slot ^ 1] = 0;
  __syncthreads();
  return all;
}

template <class T, int kVecs>
__global__ void __launch_bounds__(kThreads) scan_kernel(const BeamArgs a) {
  constexpr int kE = 16 / sizeof(T), kChunk = kThreads * kVecs;  // vectors of a chunk
  __shared__ ScanShared<kVecs> sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / a.chunks, chunk = blockIdx.x - row * a.chunks;
  if (tid == 0) sm.slots = sm.n = sm.count[0] = sm.count[1] = 0, sm.bound = -kInf;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (kind_of(a, row, a.scores[row], false) != kTokens) return;
  const T* x = static_cast<const T*>(a.logits) + row * a.stride;
  const int lead = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));  // elements before the row in its first vector
  const uint4* vecs = reinterpret_cast<const uint4*>(x - lead);
  const int v0 = chunk * kChunk + tid;
  auto token = [&](int vec, int e) { return vec * kE - lead + e; };
  auto load = [&](int vec) {
    const int p0 = token(vec, 0);
    return p0 >= 0 && p0 + kE <= a.vocab ? load_once(vecs + vec) : load_edge(x, p0, a.vocab);
  };
  uint4 v[kVecs];
  if ((lead == 0 || chunk > 0) && token((chunk + 1) * kChunk, 0) <= a.vocab) {
#pragma unroll
    for (int j = 0; j < kVecs; j++) v[j] = load_once(vecs + v0 + j * kThreads);
  } else {
#pragma unroll
    for (int j = 0; j < kVecs; j++) v[j] = load(v0 + j * kThreads);
  }
  // the chunk's largest, and the largest of its segments (of four threads each; two for long lists)
  const float mine = largest<T>(v);
  const int span = a.k > 32 ? 2 : 4, segments = kThreads / span;
  float top = fmaxf(mine, __shfl_xor_sync(~0u, mine, 1));
  if (span == 4) top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
  if (tid % span == 0) sm.segment[tid / span] = top;
#pragma unroll
  for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
  if (lane == 0) sm.top[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; w++) top = fmaxf(top, sm.top[w]);
  // a bound for the k largest: the k-th largest segment
  if (tid < segments) {
    const float u = sm.segment[tid];
    int rank = 0;
    for (int i = 0; i < segments; i += 4) {
      const float4 q = *reinterpret_cast<const float4*>(&sm.segment[i]);
      rank += (q.x > u || (q.x == u && i < tid)) + (q.y > u || (q.y == u && i + 1 < tid)) +
              (q.z > u || (q.z == u && i + 2 < tid)) + (q.w > u || (q.w == u && i + 3 < tid));
    }
    if (rank == a.k - 1) sm.bound = u;
  }
  // the sum of exponentials: exp(x - top) = 2^((x - top) log2 e)
  const float ref = top == -kInf ? 0.f : top;
  float sums[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < kVecs; j++)
    each<T>(v[j], [&](int e, float u) { sums[e & 3] += exp2_approx((u - ref) * 1.4426950408889634f); });
  float sum = (sums[0] + sums[1]) + (sums[2] + sums[3]);
#pragma unroll
  for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
  if (lane == 0) sm.sum[warp] = sum;
  __syncthreads();
  // threads with a candidate hand their vectors to whole warps
  const float bound = sm.bound;
  if (mine >= bound && mine > -kInf) {
    const int s = atomicAdd(&sm.slots, 1);
    if (s < kSlots) {
      sm.owner[s] = tid;
#pragma unroll
      for (int j = 0; j < kVecs; j++) sm.slot[s][j] = v[j];
    }
  }
  __syncthreads();
  bool fits = sm.slots <= kSlots;
  if (fits) {
    for (int s = warp; s < sm.slots; s += kWarps) {
      const T* e = reinterpret_cast<const T*>(sm.slot[s]);
      const int first = chunk * kChunk + sm.owner[s];
      for (int i = lane; i < kVecs * kE; i += 32) {
        const float u = to_float(e[i]);
        if (u >= bound && u > -kInf) {
          const int at = atomicAdd(&sm.n, 1);
          if (at < kFound) sm.found[at] = BeamItem{u + 0.f, token(first + i / kE * kThreads, i % kE)};
        }
      }
    }
    __syncthreads();
    fits = sm.n <= kFound;
  }
  if (!fits) {
    // many equal values, or all tokens that are not masked within few threads: the k-th largest exactly,
    // then of those that equal it the first ones, bit by bit.  (The logits are read again for every bit:
    // held in registers they cost the common path its occupancy.)
    int turn = 0;
    auto count = [&](auto&& f) {
      int n = 0;
#pragma unroll 1
      for (int j = 0; j < kVecs; j++) each<T>(load(v0 + j * kThreads), [&](int e, float u) { n += f(ordered(u), j, e); });
      n = block_sum(n, sm.count, turn);
      turn ^= 1;
      return n;
    };
    const uint32_t none = ordered(-kInf);
    uint32_t kth = none + 1;
    int all = count([&](uint32_t u, int, int) { return u >= kth; });
    int last = INT32_MAX;  // of the equal ones, those up to here
    if (all > a.k) {
      kth = 0;
      for (int b = 31; b >= 0; b--) {
        const uint32_t next = kth | 1u << b;
        if (count([&](uint32_t u, int, int) { return u >= next; }) >= a.k) kth = next;
      }
      const int want = a.k - count([&](uint32_t u, int, int) { return u > kth; });
      last = -1;  // (the largest position with fewer than `want` of them at or before it)
      for (int b = 14; b >= 0; b--) {
        const int next = last + (1 << b);
        if (count([&](uint32_t u, int j, int e) { return u == kth && (j * kThreads + tid) * kE + e <= next; }) < want) last = next;
      }
      last++;
    }
    if (tid == 0) sm.n = 0;
    __syncthreads();
#pragma unroll 1
    for (int j = 0; j < kVecs; j++)
      each<T>(load(v0 + j * kThreads), [&](int e, float u) {
        const uint32_t o = ordered(u);
        if (o > kth || (o == kth && (j * kThreads + tid) * kE + e <= last)) {
          const int at = atomicAdd(&sm.n, 1);
          if (at < kFound) sm.found[at] = BeamItem{u + 0.f, token(v0 + j * kThreads, e)};
        }
      });
    __syncthreads();
  }
  const int n = min(sm.n, kFound);
  const int64_t out = (int64_t)row * a.chunks + chunk;
  if (tid < n) {
    const BeamItem it = sm.found[tid];
    int rank = 0;
    for (int i = 0; i < n; i++) {
      const BeamItem o = sm.found[i];
      rank += o.logit > it.logit || (o.logit == it.logit && o.token < it.token);
    }
    if (rank < a.k) a.lists[out * a.k + rank] = it;
  }
  if (tid == 0) {
    sum = 0.f;
    for (int w = 0; w < kWarps; w++) sum += sm.sum[w];
    a.stats[out] = BeamStat{top, sum, min(n, a.k), 0};
  }
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
  if (n <= kThreads) {  // by the number of those before
    const int i = threadIdx.x;
    Place mine;
    int rank = 0;
    __syncthreads();
    if (i < n) {
      mine = p[i];
      for (int j = 0; j < n; j++) {
        const Place o = p[j];
        rank += before(o, mine) || (j < i && !before(mine, o));
      }
    }
    __syncthreads();
    if (i < n) p[rank] = mine;
    __syncthreads();
    return;
  }
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

// Chunks of a row, `vecs` vectors of `elems` logits a thread (a row may begin anywhere in its first vector).
int64_t chunks_of(int32_t vocab, int elems, int vecs) {
  return ((int64_t)vocab + elems - 1 + (int64_t)elems * kThreads * vecs - 1) / ((int64_t)elems * kThreads * vecs);
}
// Small chunks where large ones would leave SMs without work.
constexpr int kLong = 8, kShort = 2, kManyCtas = 304;
bool short_chunks(int64_t n_rows, int32_t vocab, int elems) { return n_rows * chunks_of(vocab, elems, kLong) < kManyCtas; }

template <class T>
cudaError_t launch_scan(const BeamArgs& a, bool brief, cudaStream_t stream) {
  return launch_early(brief ? scan_kernel<T, kShort> : scan_kernel<T, kLong>, dim3((unsigned)(a.n_rows * (int64_t)a.chunks)),
                      kThreads, 0, 1, stream, a);
}

}  // namespace

size_t beam_select_workspace_bytes(int64_t n_rows, int32_t vocab, int32_t k) {
  int64_t most = 1;
  for (int elems : {4, 8}) {
    // (up to n_rows rows: the short chunks of fewer rows may be more)
    const int64_t few = std::min(n_rows, (kManyCtas - 1) / chunks_of(vocab, elems, kLong));
    most = std::max({most, few * chunks_of(vocab, elems, kShort), n_rows * chunks_of(vocab, elems, kLong)});
  }
  return (size_t)most * (sizeof(BeamStat) + k * sizeof(BeamItem));
}

cudaError_t launch_beam_select(BeamArgs a, int32_t type, void* workspace, cudaStream_t stream) {
  const int elems = type == 2 ? 4 : 8;
  const bool brief = short_chunks(a.n_rows, a.vocab, elems);
  a.chunks = (int32_t)chunks_of(a.vocab, elems, brief ? kShort : kLong);
  a.stats = static_cast<BeamStat*>(workspace);
  a.lists = reinterpret_cast<BeamItem*>(a.stats + (int64_t)a.n_rows * a.chunks);
  cudaError_t e = type == 0   ? launch_scan<__nv_bfloat16>(a, brief, stream)
                  : type == 1 ? launch_scan<__half>(a, brief, stream)
                              : launch_scan<float>(a, brief, stream);
  if (e != cudaSuccess) return e;
  const int lists = a.beams * a.chunks, deep = (a.k + lists - 1) / lists;
  const size_t smem = sizeof(Place) * std::max(pow2_from(lists * deep), pow2_from(std::min(lists, a.k) * a.k));
  if (smem > 40 * 1024) {
    e = set_smem_attr_once(reinterpret_cast<const void*>(join_kernel), 128 * 1024);
    if (e != cudaSuccess) return e;
  }
  return launch_early(join_kernel, dim3(a.n_rows / a.beams), kThreads, smem, 1, stream, a);
}

}  // namespace fp4idx
