// Beam selection: the k best continuations of each group of rows (beams) over the vocabulary.
//
// total = score + (logit - lse), lse = log sum exp(logit) over the row.  Within a row the order is that
// of the logits, so the scan keeps a row's k largest logits, in lists, next to (largest, sum of exp(logit -
// largest)); the join turns these into lse and totals and picks a group's k best.
//
// Every logit is read once, and the tiles that hold a candidate once more (132 MB of 127 for wide beams): HBM bounds the
// scan while it reads (256 rows of 131,072 logits: 10 us of bf16, some 20 of fp32, 6.6 TB/s; with bf16 logits in L2, 7 us,
// it is the exponential unit).  The rest is latency: 1.5 us to the first logits, 1 us for the bound of a chunk's k largest, 2
// for reading the tiles above it again, 1 for sorting what passes, 3 to 7 for the join.  So one launch where a group fits a
// cluster, no FP64, few barriers.  64 x 4 rows of 131,072 bf16 logits take 18.0 us in all (67 MB, 3.7 TB/s), 8 x 32 of fp32
// 33.5 to 37 (127 MB, 3.4 to 3.8 TB/s), 4 rows of 32,000 7.5 to 8.3 (the host).
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "beam.cuh"
#include "mma_bf16.cuh"

namespace fp4idx {
namespace {

constexpr int kJoin = 1024;  // threads of a join by itself (8 x 32 rows 41 us against 44 with 512)
constexpr int kEarly = 2;    // candidates that a thread reads before the rows' sums are known
constexpr int kAll = 128;    // up to here a join sorts all of a group's candidates (as fast as with a bound first, which wants
                             // 32 at the least)
constexpr float kInf = __builtin_huge_valf();

__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(float v) { return v; }

// A number as the unevaluated sum of two floats, the second at most half a unit of the first (Knuth's exact
// sum of two floats; some 46 bits).  FP64 would do as well, but this GPU has next to no units for it: the
// exponentials and logarithms of a group's few sums took 3.5 to 22 us of a join in it.
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two sum_of(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return Two{s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Two operator+(const Two& a, const Two& b) {
  const Two s = sum_of(a.hi, b.hi);
  return sum_of(s.hi, __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)));
}
__device__ __forceinline__ Two operator+(const Two& a, float b) { return a + Two{b, 0.f}; }
__device__ __forceinline__ Two operator-(const Two& a) { return Two{-a.hi, -a.lo}; }
__device__ __forceinline__ Two scaled(const Two& a, float power) { return Two{a.hi * power, a.lo * power}; }
__device__ __forceinline__ Two xor_lane(const Two& a, int d) {
  return Two{__shfl_xor_sync(~0u, a.hi, d), __shfl_xor_sync(~0u, a.lo, d)};
}
// log(v) for a normal v > 0: v = 2^e f with f in [3/4, 3/2), log f = 2 artanh(s), s = (f - 1) / (f + 1) (the first
// term of its series in two floats, the others, below 0.006, in one: 7 roundings and four of sums); within 3.3e-9 (2.8e-9
// found over 40 million numbers).
__device__ __forceinline__ Two log_of(const Two& v) {
  int e = (__float_as_int(v.hi) >> 23) - 127;
  float f = __int_as_float((__float_as_int(v.hi) & 0x7FFFFF) | 0x3F800000);
  if (f >= 1.5f) f *= 0.5f, e++;
  const float n = f - 1.f;  // exact
  const Two d = sum_of(f, 1.f);
  const float s = __fdiv_rn(n, d.hi);
  const float low = (__fmaf_rn(-s, d.hi, n) - s * d.lo) / d.hi;  // of n / d
  const float z = s * s;
  const float rest = s * z * (0.33333334f + z * (0.2f + z * (0.14285715f + z * (0.11111111f + z * (0.09090909f + z * 0.07692308f)))));
  // ln 2 in two parts (Cody and Waite): the first has 16 bits, so that its product with e is exact
  const Two base = sum_of(e * 0.693145751953125f, 2.f * s);
  return base + (2.f * (low + rest) + e * 1.4286068203094173e-6f + v.lo / v.hi);
}

// What a row contributes: nothing (dead, or its score is no number), its tokens, or its end.
enum Kind : int32_t { kNone, kTokens, kEnd };
__device__ __forceinline__ Kind kind_of(const BeamArgs& a, int row, float score, bool report) {
  const bool done = a.done && a.done[row];
  if (score == -kInf) return kNone;
  if (!(score < kInf)) {  // NaN or +inf
    if (report) record_error(a.status, FP4IDX_ERR_BAD_VALUE);
    return kNone;
  }
  return done ? kEnd : kTokens;
}

// ---------------------------------------------------------------- scan
constexpr int kVecs = 4;       // vectors (16 bytes of logits) of a tile, what a thread takes at once (2 and 3: 3 % slower; 6 spills)
constexpr int kSegments = 128;  // of a chunk, half as many for lists of up to 32
constexpr int kWords = 4;      // words that a thread reads again at once
constexpr float kLog2e = 1.4426950408889634f;

template <class T>
struct Elems;
template <>
struct Elems<__nv_bfloat16> {
  static constexpr uint32_t kMasked = 0xFF80FF80u;  // -inf
  using Pair = __nv_bfloat162;
  __device__ static float2 pair(uint32_t w) { return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); }
};
template <>
struct Elems<__half> {
  static constexpr uint32_t kMasked = 0xFC00FC00u;  // -inf
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
template <class T, int kN>
__device__ __forceinline__ float largest(const uint4 (&v)[kN]) {
  if constexpr (sizeof(T) == 4) {
    float m = -kInf;
#pragma unroll
    for (int j = 0; j < kN; j++)
      m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(v[j].x), __uint_as_float(v[j].y)),
                         fmaxf(__uint_as_float(v[j].z), __uint_as_float(v[j].w))));
    return m;
  } else {
    using P = typename Elems<T>::Pair;
    uint32_t w = v[0].x;
    P m = *reinterpret_cast<P*>(&w);
#pragma unroll
    for (int j = 0; j < kN; j++)
#pragma unroll
      for (int i = j == 0; i < 4; i++) {
        uint32_t u = word_of(v[j], i);
        m = __hmax2(m, *reinterpret_cast<P*>(&u));
      }
    const float2 f = Elems<T>::pair(*reinterpret_cast<uint32_t*>(&m));
    return fmaxf(-kInf, fmaxf(f.x, f.y));
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
// Numbers in the order of their bits; larger is larger.
__device__ __forceinline__ uint32_t ordered(float v) {
  const int32_t i = __float_as_int(v + 0.f);
  return (uint32_t)i ^ (i < 0 ? 0xFFFFFFFFu : 0x80000000u);
}

__device__ __forceinline__ float unordered(uint32_t o) { return __uint_as_float(o >> 31 ? o ^ 0x80000000u : ~o); }
__host__ __device__ inline int pow2_from(int n) {
  int p = 1;
  while (p < n) p <<= 1;
  return p;
}
// Descending order; no two keys are equal.  Up to kThreads (a power of two) by counting those above each, adjacent lanes sharing one; more
// of them (a power of two) in a sorting network.
template <int kThreads>
__device__ __forceinline__ void sort_keys(uint64_t* keys, int n) {
  if (n <= kThreads) {
    const int share = min(32, kThreads / n), part = threadIdx.x & (share - 1), i = threadIdx.x / share;
    uint64_t key = 0;
    int rank = 0;
    if (i < n) {
      key = keys[i];
#pragma unroll 8
      for (int j = part; j < n; j += share) rank += keys[j] > key;
    }
#pragma unroll 1
    for (int d = 1; d < share; d <<= 1) rank += __shfl_xor_sync(~0u, rank, d);
    __syncthreads();
    if (part == 0 && i < n) keys[rank] = key;
    __syncthreads();
    return;
  }
  for (int size = 2; size <= n; size <<= 1)
    for (int d = size >> 1; d; d >>= 1) {
      for (int i = threadIdx.x; i < n / 2; i += kThreads) {
        const int lo = 2 * i - (i & (d - 1)), hi = lo + d;
        const uint64_t u = keys[lo], v = keys[hi];
        if ((v > u) == ((lo & size) == 0)) keys[lo] = v, keys[hi] = u;
      }
      __syncthreads();
    }
}

// The largest of what a thread has read, and the sum of exp(value - largest): 2^((value - largest) log2 e).
struct Running {
  float top = -kInf, sum = 0.f;

  __device__ static float ref(float m) { return m == -kInf ? 0.f : m; }
  __device__ float rescaled(float to) const { return sum * exp2_approx((top - to) * kLog2e); }
  __device__ void add(float v) {
    const float m = fmaxf(top, v);
    sum = rescaled(ref(m)) + exp2_approx((v - ref(m)) * kLog2e);
    top = m;
  }
  template <class T, int kN>
  __device__ float add(const uint4 (&v)[kN]) {  // (the largest of these)
    const float here = largest<T>(v), m = fmaxf(top, here), r = ref(m);
    uint64_t part[2] = {0, 0};
    const uint64_t minus = pack(-r, -r), scale = pack(kLog2e, kLog2e);
#pragma unroll
    for (int j = 0; j < kN; j++)
#pragma unroll
      for (int i = 0; i < 4; i += sizeof(T) / 2) {
        float2 u;
        if constexpr (sizeof(T) == 4) u = make_float2(__uint_as_float(word_of(v[j], i)), __uint_as_float(word_of(v[j], i + 1)));
        else u = Elems<T>::pair(word_of(v[j], i));
        uint64_t d = pack(u.x, u.y);
        asm("add.rn.f32x2 %0, %0, %1;\n\tmul.rn.f32x2 %0, %0, %2;" : "+l"(d) : "l"(minus), "l"(scale));
        const float2 e = unpack(d);
        asm("add.rn.f32x2 %0, %0, %1;" : "+l"(part[i >> (sizeof(T) / 4) & 1]) : "l"(pack(exp2_approx(e.x), exp2_approx(e.y))));
      }
    const float2 p = unpack(part[0]), q = unpack(part[1]);
    sum = rescaled(r) + ((p.x + p.y) + (q.x + q.y));
    top = m;
    return here;
  }
  __device__ static uint64_t pack(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
  }
  __device__ static float2 unpack(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
  }
};

template <int kThreads>
struct ScanShared {
  static constexpr int kFound = 2048;  // candidates of a chunk that are sorted
  float segment[kSegments];
  float top[kThreads / 32];
  Two sum[kThreads / 32];
  uint64_t found[kFound];  // ordered logit, then the token counted down
  int32_t owner[kThreads];  // thread + tile * kThreads
  int32_t owners, n, count[2];
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

// One chunk: its list and its sums go to `list` and `stat` (nothing, if the row has no tokens to offer).  A row's
// tokens: up to the first 16-byte boundary one by one (the head), then vectors, of which a chunk takes
// `chunk_vecs`, then the rest (the tail).  The first chunk takes the head too, the last one the tail: a list's place grows
// with its tokens, and the join takes the lower place among equal totals.  `tops` has a float for each tile of each thread;
// `begin` is called once what the launch before this one wrote may be read, `ready` by all threads before anything is
// written.
template <class T, int kThreads, class Begin, class Ready>
__device__ __forceinline__ void scan_chunk(const BeamArgs& a, int row, int chunk, ScanShared<kThreads>& sm, float* tops, BeamItem* list,
                                           BeamStat* stat, Begin&& begin, Ready&& ready) {
  constexpr int kE = 16 / sizeof(T), kWarps = kThreads / 32, kTile = kVecs * kThreads, kFound = ScanShared<kThreads>::kFound;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) sm.owners = sm.n = sm.count[0] = sm.count[1] = 0, sm.bound = -kInf;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  begin();
  if (kind_of(a, row, a.scores[row], false) != kTokens) return;
  const T* x = static_cast<const T*>(a.logits) + row * a.stride;
  const int head = min(a.vocab, (int)((16 - (reinterpret_cast<uintptr_t>(x) & 15)) % 16 / sizeof(T)));
  const int vecs = (a.vocab - head) / kE, rest = head + vecs * kE;
  const int first = min(vecs, chunk * a.chunk_vecs), end = min(vecs, first + a.chunk_vecs);
  const uint4* body = reinterpret_cast<const uint4*>(x + head);
  // this thread's token at the row's ends, -1 for none (in one expression over both ends the cluster kernels spill)
  int edge = -1;
  if (tid < 16) {
    if (chunk == 0 && tid < head) edge = tid;
    if (chunk == a.chunks - 1 && tid >= 8 && rest + tid - 8 < a.vocab) edge = rest + tid - 8;
  }
  Running run;
  // the next vectors are on their way while these are taken in
  auto load = [&](int i, uint4 (&v)[kVecs]) {
#pragma unroll
    for (int j = 0; j < kVecs; j++)
      v[j] = i + j * kThreads < end ? load_once(body + i + j * kThreads) : make_uint4(Elems<T>::kMasked, Elems<T>::kMasked, Elems<T>::kMasked, Elems<T>::kMasked);
  };
  uint4 v[2][kVecs];
  load(first + tid, v[0]);
  for (int i = first + tid, t = tid; i < end; i += 2 * kTile, t += 2 * kThreads) {
    load(i + kTile, v[1]);
    tops[t] = run.add<T>(v[0]);
    load(i + 2 * kTile, v[0]);
    if (i + kTile < end) tops[t + kThreads] = run.add<T>(v[1]);
  }
  // (earlier, the join's CTAs would take the places of CTAs of this scan that have not begun)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (edge >= 0) run.add(to_float(x[edge]));
  // the largest of all, and of segments (of adjacent threads, of fewer for long lists)
  const int segments = a.k > 32 ? kSegments : kSegments / 2, span = kThreads / segments;
  float top = run.top;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    if (d == span && (lane & (span - 1)) == 0) sm.segment[tid / span] = top;
    top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
  }
  if (lane == 0) sm.top[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; w++) top = fmaxf(top, sm.top[w]);
  Two sum{run.rescaled(Running::ref(top)), 0.f};
#pragma unroll
  for (int d = 16; d; d >>= 1) sum = sum + xor_lane(sum, d);
  if (lane == 0) sm.sum[warp] = sum;
  // a bound for the k largest: the k-th largest segment (adjacent lanes share one)
  {
    const int i = tid / span;
    const float u = sm.segment[i];
    int rank = 0;
#pragma unroll 4
    for (int s = tid & (span - 1); s < segments; s += span) {
      const float q = sm.segment[s];
      rank += (int)(q > u) | ((int)(q == u) & (int)(s < i));
    }
    for (int d = 1; d < span; d <<= 1) rank += __shfl_xor_sync(~0u, rank, d);
    if (rank == a.k - 1 && (tid & (span - 1)) == 0) sm.bound = u;
  }
  __syncthreads();
  // the tiles with a candidate are read once more, a word a thread
  const float bound = sm.bound;
  auto add = [&](uint32_t o, int token) {
    const int at = atomicAdd(&sm.n, 1);
    if (at < kFound) sm.found[at] = (uint64_t)o << 32 | (0xFFFFFFFFu - token);
  };
  auto keep = [&](float u, int token) {
    if (u >= bound && u > -kInf) add(ordered(u), token);
  };
  if (run.top >= bound && run.top > -kInf)
    for (int t = tid, i = first + tid; i < end; t += kThreads, i += kTile)
      if (tops[t] >= bound && tops[t] > -kInf) {
        const int o = atomicAdd(&sm.owners, 1);
        if (o < kThreads) sm.owner[o] = t;
      }
  if (edge >= 0) keep(to_float(x[edge]), edge);
  __syncthreads();
  const int owners = sm.owners, words = owners * kVecs * 4;
  if (owners <= kThreads) {
    for (int w = tid; w < words && *(volatile int32_t*)&sm.n <= kFound; w += kWords * kThreads) {
      uint32_t u[kWords];
      int at[kWords];  // the word's first token
#pragma unroll
      for (int j = 0; j < kWords; j++) {
        const int o = w + j * kThreads, q = o / 4 % kVecs, t = o < words ? sm.owner[o / (4 * kVecs)] : 0;
        const int i = first + t / kThreads * kTile + q * kThreads + t % kThreads;
        const bool in = o < words && i < end;
        at[j] = head + i * kE + o % 4 * (kE / 4);
        u[j] = in ? reinterpret_cast<const volatile uint32_t*>(body + i)[o % 4] : Elems<T>::kMasked;
      }
#pragma unroll
      for (int j = 0; j < kWords; j++) {
        if constexpr (kE == 4) {
          keep(__uint_as_float(u[j]), at[j]);
        } else {
          const float2 p = Elems<T>::pair(u[j]);
          keep(p.x, at[j]);
          keep(p.y, at[j] + 1);
        }
      }
    }
  }
  __syncthreads();
  if (owners > kThreads || sm.n > kFound) {
    // many equal values, or many tokens in few threads: the k-th largest exactly, then of those that equal it
    // the first ones, bit by bit
    int turn = 0;
    auto all_of = [&](auto&& f) {
      for (int v = first + tid; v < end; v += kThreads) each<T>(body[v], [&](int e, float u) { f(ordered(u), head + v * kE + e); });
      if (edge >= 0) f(ordered(to_float(x[edge])), edge);
    };
    auto count = [&](auto&& f) {
      int n = 0;
      all_of([&](uint32_t o, int token) { n += f(o, token); });
      n = block_sum(n, sm.count, turn);
      turn ^= 1;
      return n;
    };
    uint32_t kth = ordered(-kInf) + 1;
    int last = INT32_MAX;  // of the equal ones, those up to this token
    if (count([&](uint32_t o, int) { return o >= kth; }) > a.k) {
      kth = 0;
      for (int b = 31; b >= 0; b--) {
        const uint32_t next = kth | 1u << b;
        if (count([&](uint32_t o, int) { return o >= next; }) >= a.k) kth = next;
      }
      const int want = a.k - count([&](uint32_t o, int) { return o > kth; });
      last = -1;  // (the largest token with fewer than `want` of them at or before it)
      for (int b = 19; b >= 0; b--) {
        const int next = last + (1 << b);
        if (count([&](uint32_t o, int token) { return o == kth && token <= next; }) < want) last = next;
      }
      last++;
    }
    if (tid == 0) sm.n = 0;
    __syncthreads();
    all_of([&](uint32_t o, int token) {
      if (o > kth || (o == kth && token <= last)) add(o, token);
    });
    __syncthreads();
  }
  const int n = min(sm.n, kFound);
  ready();
  const int padded = pow2_from(n);
  for (int i = n + tid; i < padded; i += kThreads) sm.found[i] = i;
  __syncthreads();
  sort_keys<kThreads>(sm.found, padded);
  for (int i = tid; i < min(n, a.k); i += kThreads) {
    const uint64_t key = sm.found[i];
    list[i] = BeamItem{unordered((uint32_t)(key >> 32)), (int32_t)(0xFFFFFFFFu - (uint32_t)key)};
  }
  if (warp == kWarps - 1) {
    sum = sm.sum[lane & (kWarps - 1)];
#pragma unroll 1
    for (int d = 1; d < kWarps; d <<= 1) sum = sum + xor_lane(sum, d);
    // (of a NaN or an infinity the second float is no number)
    if (lane == 0) *stat = BeamStat{top, sum.hi, sum.hi < kInf ? sum.lo : 0.f, min(n, a.k)};
  }
}

template <class T, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) scan_kernel(const BeamArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ ScanShared<kThreads> sm;
  const int row = blockIdx.x / a.chunks;
  scan_chunk<T>(a, row, blockIdx.x - row * a.chunks, sm, reinterpret_cast<float*>(smem), a.lists + (int64_t)blockIdx.x * a.k,
                a.stats + blockIdx.x, [] {}, [] {});
}

// ---------------------------------------------------------------- join
// A group's candidates lie in shared memory list after list (beam after beam, chunk after chunk, each in order), k
// places each, kMostItems in all.  Their keys are in the order of the totals (larger is better): the first of its
// two floats, all but the last 13 bits of the second, and, so that no two keys are equal and the lower index (the lower
// row, then the lower token) comes first among equal totals, the index counted down.  What is no candidate has
// a key below 2^32.
constexpr int kIndexBits = 13, kMostItems = 1 << kIndexBits;
__device__ __forceinline__ uint64_t key_of(const Two& total, int i) {
  const uint64_t t = (uint64_t)ordered(total.hi) << 32 | ordered(total.lo);
  return (t >> kIndexBits << kIndexBits) | (kMostItems - 1 - i);
}
__device__ __forceinline__ int index_of(uint64_t key) { return kMostItems - 1 - (int)(key & (kMostItems - 1)); }
// Some 4 k candidates, and k at the least, make the bound of a join.
inline int depth(int k, int lists) {
  const int d = (4 * k + lists - 1) / lists;
  return d < k ? d : k;
}
struct JoinShared {
  // lse = top + rest, kept apart: next to a large top the sum's logarithm would be lost
  float tops[FP4IDX_BEAM_MAX_BEAMS], score[FP4IDX_BEAM_MAX_BEAMS];
  Two rest[FP4IDX_BEAM_MAX_BEAMS];
  int32_t kind[FP4IDX_BEAM_MAX_BEAMS];
  int32_t n_found;
  uint32_t bound;
};
// Where, in units of 8 bytes, the sorted keys begin (16-byte aligned): behind the keys, the tokens and the lists' sizes.
__host__ __device__ inline int sorted_at(int all, int lists) { return ((3 * all + lists + 1) / 2 + 1) & ~1; }
__host__ __device__ inline size_t join_bytes(int k, int lists) {
  const int all = lists * k;
  return sizeof(uint64_t) * (sorted_at(all, lists) + pow2_from(all));
}

// The scores of a group's rows, and what they contribute, for the thread of each row.
__device__ __forceinline__ void read_rows(const BeamArgs& a, int first, JoinShared& sm) {
  for (int b = threadIdx.x; b < a.beams; b += blockDim.x) {
    const float s = a.scores[first + b];
    sm.kind[b] = kind_of(a, first + b, s, true);
    sm.score[b] = s;
  }
}

// One group, by one CTA, from its rows' lists and sums, once read_rows has been called; `smem` has join_bytes.
template <int kThreads>
__device__ __forceinline__ void join_group(const BeamArgs& a, int group, const BeamStat* stats, const BeamItem* from,
                                           JoinShared& sm, uint8_t* smem) {
  const int tid = threadIdx.x;
  const int first = group * a.beams, k = a.k, lists = a.beams * a.chunks, all = lists * k, per_beam = a.chunks * k;
  uint64_t* keys = reinterpret_cast<uint64_t*>(smem);
  int32_t* tokens = reinterpret_cast<int32_t*>(keys + all);
  int32_t* sizes = tokens + all;
  uint64_t* sorted = keys + sorted_at(all, lists);
  if (tid == 0) sm.n_found = 0;
  BeamItem early[kEarly];  // on their way while the rows' sums are joined
#pragma unroll
  for (int j = 0; j < kEarly; j++)
    if (tid + j * kThreads < all) early[j] = from[tid + j * kThreads];
  // a row's chunks over `lanes` adjacent lanes, all of the group's rows at once if they fit
  const int lanes = a.lanes;
  __syncthreads();
  for (int b0 = 0; b0 < a.beams; b0 += kThreads / lanes) {
    const int b = b0 + tid / lanes, c0 = tid & (lanes - 1);
    const bool live = b < a.beams;
    const BeamStat* st = stats + b * a.chunks;
    // (a row without lists has what the workspace held; it is not looked at)
    BeamStat mine{-kInf, 0.f, 0.f, 0};
    if (live && c0 < a.chunks) mine = st[c0];
    int32_t what = live ? sm.kind[b] : kNone;
    float top = mine.top;
    for (int q = c0 + lanes; q < a.chunks && live; q += lanes) top = fmaxf(top, st[q].top);
    for (int d = lanes >> 1; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
    Two total{0.f, 0.f};
    for (int q = c0; q < a.chunks && live; q += lanes) {
      const BeamStat t = q == c0 ? mine : st[q];
      const float w = exp2_approx((t.top - Running::ref(top)) * kLog2e);  // (one for the chunk of the largest)
      total = total + Two{t.sum * w, t.sum_low * w};
      sizes[b * a.chunks + q] = what == kTokens ? t.count : what == kEnd && q == 0;
    }
#pragma unroll 1
    for (int d = lanes >> 1; d; d >>= 1) total = total + xor_lane(total, d);
    if (what == kTokens && !(total.hi < kInf)) {  // a logit is NaN or +inf
      if (c0 == 0) record_error(a.status, FP4IDX_ERR_BAD_VALUE);
      what = kNone;
    }
    if (what == kTokens && total.hi == 0.f) what = kNone;
    if (what == kTokens) total = log_of(total);
    if (live && c0 == 0) sm.kind[b] = what, sm.tops[b] = top, sm.rest[b] = total;
  }
  __syncthreads();
  auto put = [&](int i, BeamItem it) {
    const int l = a.by_k.under(i), b = a.by_beam.under(i);
    uint64_t key = (1 << 16) + i;
    if (sm.kind[b] != kNone && i - l * k < sizes[l]) {
      // a fourth of the total: no finite score and logits make it overflow
      Two t{sm.score[b] * 0.25f, 0.f};
      if (sm.kind[b] == kEnd) it.token = a.end_token;
      else t = sum_of(it.logit * 0.25f, sm.tops[b] * -0.25f) + -scaled(sm.rest[b], 0.25f) + t;
      key = key_of(t, i);
    }
    keys[i] = key;
    tokens[i] = it.token;
  };
#pragma unroll
  for (int j = 0; j < kEarly; j++)
    if (tid + j * kThreads < all) put(tid + j * kThreads, early[j]);
  for (int i = tid + kEarly * kThreads; i < all; i += kThreads) put(i, from[i]);
  __syncthreads();
  int n = all;
  if (all > kAll) {
    // a bound: the k-th best of each list's first `deep` candidates, by the upper bits of their totals (the index
    // in the others makes them differ); whatever is no worse in these bits stays
    const int deep = a.by_deep.d, heads = lists * deep, m = pow2_from(heads), bits = 31 - __clz(m);
    uint32_t* upper = reinterpret_cast<uint32_t*>(sorted);
    for (int i = tid; i < m; i += kThreads) {
      const int l = a.by_deep.under(i);
      const uint32_t hi = i < heads ? (uint32_t)(keys[l * k + (i - l * deep)] >> 32) : 0u;
      upper[i] = (hi >> bits << bits) | (m - 1 - i);
    }
    __syncthreads();
    const int share = max(1, min(min(32, kThreads / m), m / 4)), part = tid & (share - 1);
    for (int i = tid / share; i < m; i += kThreads / share) {  // (whole warps: m is 32 at the least)
      const uint32_t mine = upper[i];
      int rank = 0;
#pragma unroll 4
      for (int j = 4 * part; j < m; j += 4 * share) {
        const uint4 q = *reinterpret_cast<const uint4*>(upper + j);
        rank += (q.x > mine) + (q.y > mine) + (q.z > mine) + (q.w > mine);
      }
      for (int d = 1; d < share; d <<= 1) rank += __shfl_xor_sync(~0u, rank, d);
      if (rank == k - 1 && part == 0) sm.bound = max(1u, mine >> bits << bits);
    }
    __syncthreads();
    const uint32_t bound = sm.bound;
    for (int i = tid; i < all; i += kThreads) {
      const uint64_t key = keys[i];
      if ((uint32_t)(key >> 32) >= bound) sorted[atomicAdd(&sm.n_found, 1)] = key;
    }
    __syncthreads();
    n = sm.n_found;
  } else {
    for (int i = tid; i < n; i += kThreads) sorted[i] = keys[i];
  }
  const int m = pow2_from(n);
  for (int i = n + tid; i < m; i += kThreads) sorted[i] = i;
  __syncthreads();
  sort_keys<kThreads>(sorted, m);
  for (int i = tid; i < k; i += kThreads) {
    const int64_t o = (int64_t)group * k + i;
    float total = -kInf;
    int row = -1, token = -1, ended = 0;
    const uint64_t key = i < m ? sorted[i] : 0;
    if (key >> 32) {
      const int at = index_of(key), b = at / per_beam;
      total = 4.f * unordered((uint32_t)(key >> 32));
      row = first + b;
      token = tokens[at];
      ended = sm.kind[b] == kEnd || token == a.end_token;
    }
    a.out_scores[o] = total;
    a.out_rows[o] = row;
    a.out_tokens[o] = token;
    if (a.done_out) a.done_out[o] = ended;
  }
}

__global__ void __launch_bounds__(kJoin) join_kernel(const BeamArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ JoinShared sm;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t list = (int64_t)blockIdx.x * a.beams * a.chunks;
  read_rows(a, blockIdx.x * a.beams, sm);
  join_group<kJoin>(a, blockIdx.x, a.stats + list, a.lists + list * a.k, sm, smem);
}

// ---------------------------------------------------------------- both in one launch
// A cluster has a group's chunks; their lists and sums go straight to the shared memory of its first CTA, which joins
// them.
__host__ __device__ inline size_t lists_bytes(int k, int lists) {
  return (lists * (sizeof(BeamStat) + k * sizeof(BeamItem)) + 15) / 16 * 16;
}
template <class T>
__device__ __forceinline__ T* in_first_cta(T* p) {
  uint64_t r;
  asm("mapa.u64 %0, %1, 0;" : "=l"(r) : "l"(reinterpret_cast<uint64_t>(p)));
  return reinterpret_cast<T*>(r);
}
template <class T, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) select_kernel(const BeamArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ ScanShared<kThreads> scan;
  __shared__ JoinShared join;
  const int lists = a.beams * a.chunks, group = blockIdx.x / lists, list = blockIdx.x - group * lists;
  BeamStat* stats = reinterpret_cast<BeamStat*>(smem);
  BeamItem* items = reinterpret_cast<BeamItem*>(stats + lists);
  uint8_t* own = smem + lists_bytes(a.k, lists);
  // (the first CTA has to be there before it is written to)
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const int beam = list / a.chunks;
  bool waited = false;
  auto wait = [&] {
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    waited = true;
  };
  auto begin = [&] {
    if (list == 0) read_rows(a, group * a.beams, join);
  };
  scan_chunk<T>(a, group * a.beams + beam, list - beam * a.chunks, scan, reinterpret_cast<float*>(own),
                in_first_cta(items + list * a.k), in_first_cta(stats + list), begin, wait);
  if (!waited) {  // (a row that has nothing to offer)
    if (list != 0) return;
    wait();
  }
  // (only the first CTA waits: the others make room, and a barrier does not wait for threads that have ended)
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  if (list != 0) return;
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  join_group<kThreads>(a, group, stats, items, join, own);
}

// What a CTA does besides reading takes some 5 us of latency, so chunks should run at once.  Up to kWave of
// them CTAs of 512 threads take one each; above that CTAs of 256 threads (400 rows of 131,072 tokens 29 us against 37,
// 100 x 6 of 65,537 31 against 36; 256 rows of 131,072 are as fast either way), and 128 for rows of up to kSmallVecs
// vectors (1,024 rows of 10,000 tokens 17 us against 23, 1,488 rows of 842 with lists of 31 23 against 80; of 4,000
// vectors 19 either way).  kWave is two CTAs for each of this GPU's 152 SMs.  Dead rows count: 64 groups of four rows of
// 131,072 tokens, one of them alive, take 15.8 us, their live rows alone 9.7.
constexpr int kWave = 304, kSmallVecs = 2048;
// The least and the most vectors of a row that one CTA takes, what it takes to spare the join lists, and the lists that
// a join has then (one request of 8 or 16 beams 13 and 15 us, with as many chunks as SMs 25 and 27); the candidates of a
// join that more chunks do not pass (22 rows of 246,505 with lists of 44 21.5 us, 27.2 with up to 8,192; 63 rows of 204,501
// 23.4 and 26.0; 32 of 131,072 with lists of 64 24.9 and 23.0).
constexpr int kLeastVecs = 512, kMostVecs = 65536, kShortVecs = 4096, kLists = 32, kFewItems = 2048;
struct Cut {
  int32_t chunks, vecs;
  Cut(int64_t n_rows, int32_t beams, int32_t k, int32_t vocab, int elems) {
    const int64_t all = std::max(1, vocab / elems);
    const int64_t few = std::max<int64_t>(kLists / beams, all / kShortVecs);
    const int64_t want = std::max<int64_t>(1, std::min({kWave / n_rows, (int64_t)(kFewItems / (beams * k)), few}));
    int64_t each = std::max<int64_t>(kLeastVecs, (all + want - 1) / want);
    each = std::min<int64_t>((each + 31) / 32 * 32, kMostVecs);
    vecs = (int32_t)each;
    chunks = (int32_t)((all + each - 1) / each);
  }
};

// Chunks of a row in a cluster of a group: no more CTAs than run at once, or one.  The cluster spares a launch (64 x 4
// rows 18.1 us against 19.7) and is taken for up to kSlack vectors more a CTA (16 x 5 rows of 50,001 8.9 us against 11.1).
constexpr int kMaxCluster = 8, kSlack = 8192;
constexpr size_t kSelectSmem = 100 * 1024;
int32_t cluster_chunks(int64_t n_rows, int32_t beams) {
  return (int32_t)std::min<int64_t>(kMaxCluster / beams, std::max<int64_t>(1, kWave / n_rows));
}

template <class T, int kThreads>
cudaError_t launch_scan(BeamArgs a, bool cluster, cudaStream_t stream) {
  const int lists = a.beams * a.chunks;
  a.by_k = Divisor(a.k);
  a.by_beam = Divisor(a.chunks * a.k);
  a.by_deep = Divisor(depth(a.k, lists));
  a.lanes = std::min(32, pow2_from(a.chunks));
  const dim3 grid((unsigned)(a.n_rows * (int64_t)a.chunks));
  const size_t tops = sizeof(float) * kThreads * ((a.chunk_vecs + kVecs * kThreads - 1) / (kVecs * kThreads));
  cudaError_t e;
  if (cluster) {
    e = set_smem_attr_once(reinterpret_cast<const void*>(select_kernel<T, kThreads>), kSelectSmem);
    if (e != cudaSuccess) return e;
    return launch_early(select_kernel<T, kThreads>, grid, kThreads, lists_bytes(a.k, lists) + std::max(tops, join_bytes(a.k, lists)),
                        lists, stream, a);
  }
  e = set_smem_attr_once(reinterpret_cast<const void*>(scan_kernel<T, kThreads>), sizeof(float) * kMostVecs / kVecs);
  if (e == cudaSuccess) e = set_smem_attr_once(reinterpret_cast<const void*>(join_kernel), 168 * 1024);
  if (e == cudaSuccess) e = launch_early(scan_kernel<T, kThreads>, grid, kThreads, tops, 1, stream, a);
  if (e != cudaSuccess) return e;
  return launch_early(join_kernel, dim3(a.n_rows / a.beams), kJoin, join_bytes(a.k, lists), 1, stream, a);
}

template <class T>
cudaError_t launch_typed(BeamArgs a, cudaStream_t stream) {
  const Cut cut(a.n_rows, a.beams, a.k, a.vocab, 16 / sizeof(T));
  a.chunks = cut.chunks;
  a.chunk_vecs = cut.vecs;
  // one launch where a group's rows fit a cluster, and its CTAs have little more to read each
  const int64_t each = cluster_chunks(a.n_rows, a.beams), all = std::max<int64_t>(1, a.vocab / (16 / sizeof(T)));
  bool cluster = false;
  if (each > 0) {
    const int64_t vecs = std::max<int64_t>(kLeastVecs, ((all + each - 1) / each + 31) / 32 * 32);
    cluster = vecs <= std::min(cut.vecs + kSlack, kMostVecs);
    if (cluster) {
      a.chunk_vecs = (int32_t)vecs;
      a.chunks = (int32_t)((all + vecs - 1) / vecs);
    }
  }
  a.lists = reinterpret_cast<BeamItem*>(a.stats + (int64_t)a.n_rows * a.chunks);
  if ((int64_t)a.n_rows * a.chunks <= kWave) return launch_scan<T, 512>(a, cluster, stream);
  return a.chunk_vecs > kSmallVecs ? launch_scan<T, 256>(a, cluster, stream) : launch_scan<T, 128>(a, cluster, stream);
}

}  // namespace

size_t beam_select_workspace_bytes(int64_t n_rows, int32_t vocab, int32_t k) {
  // enough for up to n_rows rows of any type (of fewer rows each may have more chunks)
  int64_t most = 1;
  for (int elems : {4, 8}) {
    const int64_t all = std::max(1, vocab / elems), least = (all + kMostVecs - 1) / kMostVecs;
    most = std::max(most, std::min(n_rows * ((all + kLeastVecs - 1) / kLeastVecs), std::max<int64_t>(kWave, n_rows * least)));
  }
  return (size_t)most * (sizeof(BeamStat) + k * sizeof(BeamItem));
}

cudaError_t launch_beam_select(BeamArgs a, int32_t type, void* workspace, cudaStream_t stream) {
  a.stats = static_cast<BeamStat*>(workspace);
  return type == 0   ? launch_typed<__nv_bfloat16>(a, stream)
         : type == 1 ? launch_typed<__half>(a, stream)
                     : launch_typed<float>(a, stream);
}

}  // namespace fp4idx
