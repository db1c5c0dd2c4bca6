// Absorbed latent attention on the tensor cores: one latent row a token is the key of every
// head (all its dims) and their value (its first 512).
//
//   S^T[tokens, columns] = K Q^T            M = 64 tokens, N = columns, K = width
//   P^T = exp2(c S^T - m)                   c = scale log2(e), m: the columns' reference
//   O^T[dims, columns] += V^T P^T           M = 128 dims (four times), N = columns, K = 64
//
// A column is a (row, head) pair; up to 64 share a pass over the tokens.  The transposed form
// keeps the tensor cores' M full with tokens and dims however few the heads are, and lets
// the same bytes in shared memory be both operands: a tile of 64 tokens is loaded once, as
// 128-byte-swizzled blocks of 64 dims, which the first product reads with K = dims contiguous
// and the second with M = dims contiguous.
//
// One persistent CTA an SM:
//   warps 0-3   (0-7 with 64 columns, half of them each) softmax: S^T from tensor memory,
//               masks, exp2, P^T to shared memory; at the end of a segment the output
//   then two warps that issue the MMAs of either product,
//   a warp      that copies a segment's queries (boxes by TMA where the columns are adjacent rows
//               of q, else 16 bytes a lane),
//   a warp      that walks kAhead tiles ahead of the softmax and prefetches their tokens into L2,
//               so that two stages in shared memory suffice to stream from HBM
//   the others  groups of four warps, one per stage, copy tiles: whole pages by TMA, listed
//               tokens and partial pages with 16-byte cp.async (tokens that no row sees become
//               zero rows)
// A unit is one row, or adjacent rows of a sequence, and up to 64 columns.  Few units get a
// cluster or a CTA each; else the list of all units' tiles is cut into runs of tiles, one a CTA,
// whatever the lengths are.  A unit cut between CTAs leaves each piece's unnormalised output,
// maximum and sum in the workspace; combine_kernel joins them in order.  All joins add in a
// fixed order: the same bits every time.
//
// What bounds it, at the sizes measured (a plain copy reaches 6.8 TB/s):
//   whole contexts, 16 heads, width 576   HBM: 64 sequences of up to 16,384 tokens, 673 MB in
//               128 us, 5.3 TB/s
//   64 columns (selections with 64 heads, trees)   shared memory: a tile takes 2,650 cycles, of
//               which 2,500 are its operands' bytes at 128 a cycle: keys and queries for the
//               scores (M = 64 re-reads the queries every tile) 1,152, values and four times the
//               weights 768, the tile's arrival 576.  1,536 selections of 2,048 tokens, 64 heads,
//               width 576: 496 to 507 us
//   few rows    latency: launch, lengths, list, pages and tokens are dependent reads, some 8 us;
//               one row of 64 heads over 512 tokens 11.7 us
//
// The reference m of a column is not its running maximum: it is only raised when a score
// passes it by more than 8 (in powers of two), so that in nearly all tiles the output in
// tensor memory needs no rescaling and the warps exchange one vote.  The result does not
// depend on m, up to rounding; weights stay below 2^8.
#include <algorithm>
#include <cmath>

#include "latent.cuh"
#include "mma_bf16.cuh"
#include "pipeline.cuh"

namespace fp4idx {
namespace {

using pipe::Ctl;
using pipe::kFull;

constexpr int kTile = 64;         // tokens a tile: one page
constexpr int kMaxCtas = 160;     // slots of the workspace
constexpr int kCols = 64;         // columns of a workspace slot
constexpr int kValue = FP4IDX_LATENT_VALUE;
// roles behind the softmax warps
constexpr int kScoreRole = 0, kOutRole = 1, kQueryRole = 2, kAheadRole = 3, kLoadRole = 4;
constexpr uint32_t kAhead = 3;    // tiles that the prefetches are ahead of the softmax
constexpr int kMaxGroup = 8;      // rows a unit
constexpr float kRaise = 8.f;
constexpr float kNoMax = -3.0e38f;

struct Params {
  LatentArgs a;
  int32_t hb, hs, hp, group;  // head blocks, heads a block, heads a block padded to 8, rows a unit at most
  int32_t q_boxes;            // a unit's columns are adjacent rows of q: copied as boxes
  int32_t whole;              // selected rows: CTAs take whole units, one after the other
  int32_t cluster;            // CTAs (a cluster, if more than one) that share a unit; 0: the list is cut
  uint64_t wait_limit_ns;
  int32_t idle_producers;
};

// Workspace: per slot (two a CTA) a record, the columns' m and l, and the output.
struct Record {
  int32_t r0, rows, hb, flags;
};
constexpr int kBegins = 1, kEnds = 2, kUsed = 4;
struct Work {
  Record* rec;
  float* ml;
  float* o;
  uint32_t* taken;  // units that CTAs have asked for (zero before a launch that counts)
};
__host__ __device__ __forceinline__ Work work_view(void* ws) {
  uint8_t* p = reinterpret_cast<uint8_t*>(ws);
  Work w;
  w.rec = reinterpret_cast<Record*>(p);
  w.ml = reinterpret_cast<float*>(p + 2 * kMaxCtas * sizeof(Record));
  w.o = w.ml + 2 * kMaxCtas * 2 * kCols;
  w.taken = reinterpret_cast<uint32_t*>(w.o + (size_t)2 * kMaxCtas * kCols * kValue);
  return w;
}
constexpr size_t kWorkBytes =
    2 * kMaxCtas * (sizeof(Record) + 2 * kCols * sizeof(float) + (size_t)kCols * kValue * sizeof(float)) + 128;

// ---------------------------------------------------------------- the list of tiles
// Row t's sequence and the tokens that it sees: its plain length, and the end of what it sees
// (0, 0: nothing).  All loads are in flight together.
template <bool kSelected>
__device__ __forceinline__ void row_span(const LatentArgs& a, int t, int& seq, int& len, int& end, int& err) {
  seq = a.row_seq[t];
  const int n = kSelected && !a.context_lens ? a.k : a.context_lens[t];
  int extra = 0;
  if (!kSelected) {
#pragma unroll
    for (int w = 0; w < FP4IDX_LATENT_MAX_TREE_WORDS; w++) {
      const uint32_t m = w < a.words ? a.tree[(int64_t)t * a.words + w] : 0;
      if (m) extra = 32 * w + 32 - __clz(m);
    }
  }
  len = end = 0;
  if (seq < 0 || seq >= a.num_seqs) {
    err = FP4IDX_ERR_BAD_PAGE;
  } else if (kSelected) {
    len = end = max(0, min(a.k, n));
  } else if (n < 0 || (int64_t)n + extra > a.max_context) {
    err = FP4IDX_ERR_BAD_LENGTH;
  } else {
    len = n;
    end = n + extra;
  }
}
// (an empty unit still writes its zeros)
__device__ __forceinline__ int tiles_of(int end) { return max(1, (end + kTile - 1) / kTile); }

// The unit that starts at row r0: adjacent rows of one sequence, up to p.group.
struct Unit {
  int r0, rows, seq, tiles;
  int min_len;   // every row sees the tokens before it
  int len, end;  // of row r0 + lane
};
// By a warp, a row a lane (one after the other, eight rows cost eight times the latency of a load).
template <bool kSelected>
__device__ __forceinline__ void load_unit(const Params& p, int r0, Unit& u, bool report) {
  const int lane = threadIdx.x & 31;
  const bool mine = lane < (kSelected ? 1 : p.group) && r0 + lane < p.a.n_rows;
  int seq = 0, len = 0, end = 0, err = 0;
  if (mine) row_span<kSelected>(p.a, r0 + lane, seq, len, end, err);
  u.r0 = r0;
  u.seq = __shfl_sync(kFull, seq, 0);
  u.rows = kSelected ? 1 : __ffs(~__ballot_sync(kFull, mine && seq == u.seq)) - 1;
  const bool in = lane < u.rows;
  if (err && in && report) record_error(p.a.status, err);
  u.len = len;
  u.end = end;
  u.min_len = __reduce_min_sync(kFull, in ? len : INT32_MAX);
  u.tiles = tiles_of(__reduce_max_sync(kFull, in ? end : 0));
}

// A run of tiles [t0, t1) of a unit's column block.
constexpr int kEnd = 3;  // tiles that the end of a unit, its output and the next one's start cost
struct Seg {
  Unit u;
  int hb, t0, t1;
  int64_t left;  // tiles of the CTA from t0 on, and kEnd for each unit that ends
  uint32_t n;    // segments of the CTA before this one
};
// Whole units: the first warp of a CTA that needs the next one (a loader) asks for it and passes it
// on through a ring in shared memory: (segment's number, unit; kNoUnit behind the last).  The
// loaders look at most four times three tiles ahead of the slowest warp, so entries are not
// overtaken, but for the prefetches', which then stop.
constexpr uint32_t kFeed = 32, kNoUnit = ~0u;
struct Feed {
  volatile uint64_t* ring;
  uint32_t* asked;  // segments asked for
  Ctl ctl;
};
template <bool kSelected, bool kShared>
__device__ __forceinline__ bool next_seg(const Params& p, Seg& s, const Feed& feed, bool report = false) {
  if (kShared) return false;  // one segment a unit
  if (kSelected && p.whole) {
    const uint32_t n = ++s.n;
    uint32_t u = kNoUnit;
    if ((threadIdx.x & 31) == 0) {
      if (atomicCAS(feed.asked, n - 1, n) == n - 1) {
        u = gridDim.x + atomicAdd(work_view(p.a.workspace).taken, 1u);
        if (u >= (uint32_t)(p.a.n_rows * p.hb)) u = kNoUnit;
        feed.ring[n % kFeed] = (uint64_t)n << 32 | u;
      } else {
        const int64_t t0 = clock64();
        uint64_t got;
        while ((uint32_t)((got = feed.ring[n % kFeed]) >> 32) < n) {
          if (*feed.ctl.abort) break;
          if (clock64() - t0 > (int64_t)feed.ctl.timeout_ns) {
            pipe::give_up(feed.ctl);
            break;
          }
        }
        if ((uint32_t)(got >> 32) == n) u = (uint32_t)got;
      }
    }
    u = __shfl_sync(kFull, u, 0);
    if (u == kNoUnit) return false;
    s.hb = (int)(u % p.hb);
    load_unit<kSelected>(p, (int)(u / p.hb), s.u, report);
    s.t0 = 0;
    s.t1 = s.u.tiles;
    return true;
  }
  s.left -= s.t1 - s.t0 + (s.t1 == s.u.tiles ? kEnd : 0);
  if (s.left <= 0) return false;
  if (++s.hb == p.hb) {
    s.hb = 0;
    load_unit<kSelected>(p, s.u.r0 + s.u.rows, s.u, false);
  }
  s.t0 = 0;
  s.t1 = (int)min((int64_t)s.u.tiles, s.left);
  return true;
}

// ---------------------------------------------------------------- the CTA's run
// All threads find the CTA's first unit and tile.  Rows are taken blockDim.x at a time.
//
// Up to one unit a CTA, where that balances: each unit gets CTAs of its own, as many as it
// takes for no CTA to have more than `most` tiles.  A CTA then has one piece, and 64 units of
// 32 tiles make 128 pieces for the joining kernel instead of the 304 of an even cut over 152
// CTAs (a piece's end costs as much as two tiles, and its 128 KB are written and read again).
// Taken when `most` is at most an even share plus 1/16 and three tiles.
// Few units: a cluster of up to 16 CTAs shares a unit and adds its pieces up through distributed
// shared memory, or one CTA takes it.  There is no workspace and no second launch then, and
// no scan where units are single rows; together these cost what six to nine tiles do (rows of
// 12 to 128 heads over 9 to 20 tiles: 30.2 us against 36.3, 21.6 against 25.6, 15.6 against
// 22.6), so this form is taken while a CTA gets at most kMore tiles above an even share.  Whole
// contexts differ in length, and the host knows only the longest that may come: the list
// is cut evenly above kMost tiles a CTA.
// More units, of rows with a selection each: the CTAs take whole units in order, each the next
// one when it needs one.  No pieces, and the rows of one sequence, whose selections overlap,
// are read at the same time (L2 then holds what they share).  1,488 units of 2,048 tokens: 655
// us by an even cut, 496 so; 360 of 500 tokens and two head blocks 106 and 83; 384 of 2,048
// 162 and 149.  With less than two units a CTA only where the last round adds at most kMore
// tiles (235 of 1,667: 92 us either way).
// Otherwise the list of tiles is cut evenly, a unit's end counting as kEnd tiles (without that, a
// CTA with 19 empty units took 122 us where the others took 65), and a cut within 1/20 of a run
// from a unit's edge moves to the edge (no piece then, for 1/20 more work).
constexpr int kMore = 8, kMost = 32;
constexpr int kMaxWarps = 20;
struct ScanShared {
  int64_t sums[kMaxWarps];
  int32_t starts[kMaxWarps];
  int32_t enough[kMaxWarps];
  int32_t tiles[kMaxWarps * 32], seqs[kMaxWarps * 32], ends[kMaxWarps * 32];
  int32_t found_row, found_hb, found_t0, found_left;
  int64_t cut[2];
};
struct Weight {
  int32_t tiles, rows;  // of the unit that starts at the thread's row; 0 tiles: none does
};
__device__ __forceinline__ int64_t weight_of(const Weight& w) { return w.tiles ? w.tiles + kEnd : 0; }
__device__ __forceinline__ int64_t block_scan(int64_t v, ScanShared& sh, int64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t u = __shfl_up_sync(kFull, v, d);
    if (lane >= d) v += u;
  }
  if (lane == 31) sh.sums[warp] = v;
  __syncthreads();
  int64_t s = lane < warps ? sh.sums[lane] : 0;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t u = __shfl_up_sync(kFull, s, d);
    if (lane >= d) s += u;
  }
  total = __shfl_sync(kFull, s, 31);
  const int64_t before = __shfl_sync(kFull, s, (warp + 31) & 31);
  __syncthreads();
  return (warp ? before : 0) + v;
}
// `run` carries the first row of the last run of one sequence from chunk to chunk.
template <bool kSelected>
__device__ __forceinline__ Weight unit_weight(const Params& p, int base, int& run, ScanShared& sh, bool report) {
  const int t = base + (int)threadIdx.x;
  const bool in = t < p.a.n_rows;
  const bool grouped = !kSelected && p.group > 1;
  int seq = 0, len, end = 0, err = 0;
  if (in) row_span<kSelected>(p.a, t, seq, len, end, err);
  if (err && report) record_error(p.a.status, err);
  if (!grouped) return in ? Weight{tiles_of(end), 1} : Weight{0, 0};
  const int before = in && t > 0 ? p.a.row_seq[t - 1] : 0;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int first = in && (t == 0 || seq != before) ? t : -1;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int u = __shfl_up_sync(kFull, first, d);
    if (lane >= d) first = max(first, u);
  }
  if (lane == 31) sh.starts[warp] = first;
  sh.seqs[threadIdx.x] = seq;
  sh.ends[threadIdx.x] = end;
  __syncthreads();
  int last = run;
  for (int w = 0; w < warps; w++) {
    if (w < warp) first = max(first, sh.starts[w]);
    last = max(last, sh.starts[w]);
  }
  first = max(first, run);
  Weight got{0, 0};
  if (in && (t - first) % p.group == 0) {
    int rows = 1;
    for (; rows < p.group && t + rows < p.a.n_rows; rows++) {
      int seq1, len1, end1, err1;
      const int at = (int)threadIdx.x + rows;
      if (at < (int)blockDim.x) {
        seq1 = sh.seqs[at];
        end1 = sh.ends[at];
      } else {  // of the next chunk
        row_span<kSelected>(p.a, t + rows, seq1, len1, end1, err1);
      }
      if (seq1 != seq) break;
      end = max(end, end1);
    }
    got = Weight{tiles_of(end), rows};
  }
  __syncthreads();
  run = last;
  return got;
}
template <bool kSelected, bool kShared>
__device__ __forceinline__ bool first_seg(const Params& p, Seg& s, ScanShared& sh, int& u) {
  const int n = p.a.n_rows, step = blockDim.x;
  if (kShared) {
    const int j = blockIdx.x & (p.cluster - 1);
    int row = u / p.hb;
    s.hb = u % p.hb;
    if (!kSelected && p.group > 1) {
      // the u-th unit's first row (all rows are one chunk here), and the cluster's next unit
      int run = -1;
      int64_t units;
      const Weight w = unit_weight<kSelected>(p, 0, run, sh, false);
      const int64_t at = block_scan(w.tiles > 0, sh, units);
      if (w.tiles > 0 && at == u + 1) sh.found_row = threadIdx.x;
      __syncthreads();
      if (u >= units) {  // fewer units than clusters
        u = -1;
        s.u.rows = s.u.r0 = 0;
        return false;
      }
      u += gridDim.x >> (__ffs(p.cluster) - 1);
      if (u >= units) u = -1;
      row = sh.found_row;
      s.hb = 0;
    } else {
      u = -1;
    }
    load_unit<kSelected>(p, row, s.u, threadIdx.x < 32 && j == 0);
    s.t0 = (int)((int64_t)s.u.tiles * j / p.cluster);
    s.t1 = (int)((int64_t)s.u.tiles * (j + 1) / p.cluster);
    s.left = s.t1 - s.t0;
    return s.left > 0;
  }
  if (kSelected && p.whole) {
    const int u = blockIdx.x;
    load_unit<kSelected>(p, u / p.hb, s.u, threadIdx.x < 32);
    s.hb = u % p.hb;
    s.t0 = 0;
    s.t1 = s.u.tiles;
    return true;
  }
  const bool report = blockIdx.x == 0;
  int64_t all = 0, incl = 0, total;
  int run = -1;
  Weight w{0, 0};
  for (int base = 0; base < n; base += step) {
    w = unit_weight<kSelected>(p, base, run, sh, report);
    incl = block_scan(weight_of(w) * p.hb, sh, total);
    all += total;
  }
  const int ctas = gridDim.x, cta = blockIdx.x;
  if (n <= step) {
    sh.tiles[threadIdx.x] = w.tiles;
    const int units = __syncthreads_count(w.tiles > 0) * p.hb;
    if (units <= ctas) {
      // each warp tries one number of tiles a CTA
      const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = step >> 5;
      const int64_t tiles = all - (int64_t)kEnd * units;
      const int least = (int)((tiles + ctas - 1) / ctas), span = (int)(tiles / ctas / 16) + 3;
      const int gap = (span + warps - 1) / warps;
      const int mine = least + warp * gap;
      int need = 0;
      for (int t = lane; t < n; t += 32) need += (sh.tiles[t] + mine - 1) / mine;
      need = __reduce_add_sync(kFull, need) * p.hb;
      if (lane == 0) sh.enough[warp] = need <= ctas;
      __syncthreads();
      const uint32_t yes = __ballot_sync(kFull, lane < warps && sh.enough[lane]);
      if (yes) {
        const int most = least + (__ffs(yes) - 1) * gap;
        const int per = (w.tiles + most - 1) / most;
        const int64_t end = block_scan((int64_t)per * p.hb, sh, total), begin = end - (int64_t)per * p.hb;
        if (cta >= total) return false;
        if (cta >= begin && cta < end) {
          const int k = cta - (int)begin, j = k % per;
          sh.found_row = (int)threadIdx.x;
          sh.found_hb = k / per;
          sh.found_t0 = (int)((int64_t)w.tiles * j / per);
          sh.found_left = (int)((int64_t)w.tiles * (j + 1) / per) - sh.found_t0;
        }
        __syncthreads();
        load_unit<kSelected>(p, sh.found_row, s.u, false);
        s.hb = sh.found_hb;
        s.t0 = sh.found_t0;
        s.left = sh.found_left;
        s.t1 = s.t0 + sh.found_left;
        return true;
      }
    }
  }
  if (threadIdx.x == 0) sh.cut[1] = all;
  const int64_t x0 = all * cta / ctas, x1 = all * (cta + 1) / ctas, near = all / ctas / 20;
  int64_t carry = 0;
  run = -1;
  __syncthreads();
  for (int base = 0; base < n; base += step) {
    if (n > step) {
      w = unit_weight<kSelected>(p, base, run, sh, false);
      incl = block_scan(weight_of(w) * p.hb, sh, total);
    }
    const int64_t weight = weight_of(w), end = carry + incl, begin = end - weight * p.hb;
#pragma unroll
    for (int i = 0; i < 2; i++) {
      int64_t x = i ? x1 : x0;
      if (x < begin || x >= end) continue;
      const int off = (int)((x - begin) % weight);
      if (off <= near) x -= off;
      else if (weight - off <= near + kEnd) x += weight - off;
      sh.cut[i] = x;
      if (i == 0) {
        const int64_t at = x - begin;
        const bool past = x == end;
        sh.found_row = base + (int)threadIdx.x + (past ? w.rows : 0);
        sh.found_hb = past ? 0 : (int)(at / weight);
        sh.found_t0 = past ? 0 : (int)(at % weight);
      }
    }
    carry += total;
    if (x1 < carry) break;
  }
  __syncthreads();
  s.left = sh.cut[1] - sh.cut[0];
  if (s.left <= 0) return false;
  load_unit<kSelected>(p, sh.found_row, s.u, false);
  s.hb = sh.found_hb;
  s.t0 = sh.found_t0;
  s.t1 = (int)min((int64_t)s.u.tiles, s.t0 + s.left);
  return true;
}

// One arrival for the warp's writes (each lane has fenced its own): an arrival of every lane
// is an atomic on one word each.
__device__ __forceinline__ void arrive_warp(uint32_t bar, int lane) {
  __syncwarp();
  if (lane == 0) ptx::mbar_arrive(bar);
}

// ---------------------------------------------------------------- shared memory
template <int kWidth, int kN>
struct Shape {
  static constexpr int kChunks = kWidth / 64;
  static constexpr uint32_t kStageBytes = kChunks * kTile * 128;
  static constexpr uint32_t kQChunk = kN * 128;
  // The weights have a buffer a stage, so that a tile's softmax does not wait for the last
  // tile's second product.  At width 576 it is the stage's last block of keys, which only the
  // first product reads; at width 512 it lies behind the queries.
  static constexpr bool kOwnP = kChunks == 8;
  // a third stage where it fits (width 512 with at most 16 columns)
  static constexpr int kStages = 3 * (kStageBytes + kQChunk) + kChunks * kQChunk <= 225 * 1024 && kOwnP ? 3 : 2;
  static constexpr int kSoftWarps = kN == 64 ? 8 : 4;
  static constexpr int kScoreWarp = kSoftWarps + kScoreRole, kOutWarp = kSoftWarps + kOutRole;
  static constexpr int kQueryWarp = kSoftWarps + kQueryRole;
  static constexpr int kAheadWarp = kSoftWarps + kAheadRole, kLoadWarp = kSoftWarps + kLoadRole;
  static constexpr int kThreads = (kLoadWarp + 4 * kStages) * 32;
  static constexpr uint32_t kOffQ = kStages * kStageBytes;
  static constexpr uint32_t kOffP = kOffQ + kChunks * kQChunk;
  static constexpr uint32_t kOffSeen = kOffP + (kOwnP ? kStages * kQChunk : 0);          // [stage][64] rows that see the token
  static constexpr uint32_t kOffRed = kOffSeen + kStages * kTile;  // [4][kN] floats
  static constexpr uint32_t kOffM = kOffRed + 4 * kN * 4;          // [kN]
  static constexpr uint32_t kOffF = kOffM + kN * 4;                // [kN]
  static constexpr uint32_t kOffBar = kOffF + kN * 4;
  // kfull[stages][2], kempty[stages][2], qfull, qempty, sfull[2], pfull[2], done
  static constexpr int kBars = 4 * kStages + 7;
  static constexpr uint32_t kOffMisc = kOffBar + kBars * 8;
  static constexpr uint32_t kOffFeed = kOffMisc + 16;
  static constexpr uint32_t kBytes = kOffFeed + kFeed * 8 + 1024;  // and the base's alignment
  static_assert(kQChunk <= kTile * 128, "the weights fit a block of keys");
  static __device__ __forceinline__ uint32_t off_p(int stage) {
    return kOwnP ? kOffP + stage * kQChunk : stage * kStageBytes + 8 * kTile * 128;
  }
  static constexpr uint32_t kTmemCols = kN == 64 ? 512 : kN == 32 ? 256 : 128;
};
// The scan's scratch lies in the query buffer, which is not in use yet.

// kShared: a cluster or a CTA a unit, joined here.  (A kernel of its own: with both forms in one, one
// long sequence took 48.4 us instead of 47.4, trees of 13 drafts 132.8 instead of 130.5, a batch of
// whole contexts 129.7 instead of 127.7, one selected row 12.3 instead of 11.6.)
template <int kWidth, int kN, bool kSelected, bool kShared>
__global__ void __launch_bounds__(Shape<kWidth, kN>::kThreads, 1) latent_attn_kernel(const __grid_constant__ CUtensorMap cache_map,
                                                                                   const __grid_constant__ CUtensorMap q_map,
                                                                                   const __grid_constant__ Params p) {
  using S = Shape<kWidth, kN>;
  constexpr int kStages = S::kStages, kChunks = S::kChunks, kSoft = S::kSoftWarps * 32;
  constexpr int kScoreWarp = S::kScoreWarp, kOutWarp = S::kOutWarp, kQueryWarp = S::kQueryWarp;
  constexpr int kAheadWarp = S::kAheadWarp, kLoadWarp = S::kLoadWarp;
  constexpr int kMyCols = kN * 4 / S::kSoftWarps, kJ = kMyCols / 8;  // columns of a softmax warp
  extern __shared__ uint8_t smem_raw[];
  const LatentArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t raw = ptx::smem_addr(smem_raw);
  uint8_t* smem = smem_raw + ((1024 - (raw & 1023)) & 1023);
  const uint32_t sb = ptx::smem_addr(smem);

  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(smem + S::kOffMisc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kOffMisc + 4);
  volatile uint64_t* feed_ring = reinterpret_cast<volatile uint64_t*>(smem + S::kOffFeed);
  auto bar = [&](int i) { return sb + S::kOffBar + i * 8; };
  // A stage is filled and freed in two halves, dims 0..255 and the rest, so that the scores'
  // product begins while the second half is on its way, and the next tile's first half is
  // copied while the output's second half is computed.
  const auto kfull = [&](int s, int half) { return bar(2 * s + half); };
  const auto kempty = [&](int s, int half) { return bar(2 * (kStages + s) + half); };
  const uint32_t qfull = bar(4 * kStages), qempty = bar(4 * kStages + 1), done = bar(4 * kStages + 6);
  const auto sfull = [&](int b) { return bar(4 * kStages + 2 + b); };
  const auto pfull = [&](int b) { return bar(4 * kStages + 4 + b); };  // by the tile's parity, as sfull
  const auto init_barriers = [&]() {
    for (int s = 0; s < kStages; s++) {
      for (int half = 0; half < 2; half++) {
        ptx::mbar_init(kfull(s, half), 4);
        ptx::mbar_init(kempty(s, half), 1);
      }
    }
    ptx::mbar_init(qfull, 1);
    ptx::mbar_init(qempty, 1);
    ptx::mbar_init(sfull(0), 1);
    ptx::mbar_init(sfull(1), 1);
    ptx::mbar_init(pfull(0), S::kSoftWarps);
    ptx::mbar_init(pfull(1), S::kSoftWarps);
    ptx::mbar_init(done, 2);
    *reinterpret_cast<volatile uint32_t*>(smem + S::kOffMisc + 8) = 0;  // tiles that the softmax has begun
    ptx::fence_mbar_init();
  };
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (uint32_t i = 0; i < kFeed; i++) feed_ring[i] = 0;
    *reinterpret_cast<volatile uint32_t*>(smem + S::kOffMisc + 12) = 0;
    init_barriers();
  }
  if (warp == kScoreWarp) ptx::tmem_alloc(ptx::smem_addr(tmem_slot), S::kTmemCols);
  // Lists, page table and queries into L2, a line a thread of the whole grid, while the run is
  // being found: three dependent reads lie between the lengths and the first tile.
  {
    const int64_t at = ((int64_t)blockIdx.x * S::kThreads + threadIdx.x) * 128;
    if (kSelected && at < (int64_t)a.n_rows * a.k * 4) pipe::prefetch_l2(reinterpret_cast<const uint8_t*>(a.idx) + at);
    if (at < (int64_t)a.num_seqs * a.max_pages * 4) pipe::prefetch_l2(reinterpret_cast<const uint8_t*>(a.page_table) + at);
    if (at < (int64_t)a.n_rows * a.heads * (kWidth * 2)) pipe::prefetch_l2(reinterpret_cast<const uint8_t*>(a.q) + at);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int cluster = kShared ? p.cluster : 0;
  int unit = kShared ? (int)blockIdx.x >> (__ffs(cluster) - 1) : -1;
  bool gave_up = false;
again:  // (clusters take unit after unit if a call has more than the host counts on)
  Seg seg;
  seg.n = 0;
  const bool any = first_seg<kSelected, kShared>(p, seg, *reinterpret_cast<ScanShared*>(smem + S::kOffQ), unit) && !gave_up;
  Work wk = work_view(a.workspace);
  if (threadIdx.x == 0 && !kShared) {
    wk.rec[2 * blockIdx.x] = Record{0, 0, 0, 0};
    wk.rec[2 * blockIdx.x + 1] = Record{0, 0, 0, 0};
  }
  ptx::fence_proxy_async_smem();  // the scratch lies where queries will be copied to
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Ctl ctl{abort_flag, a.status, 2 * p.wait_limit_ns};  // in cycles: at most 2.07 a ns
  const Feed feed{feed_ring, reinterpret_cast<uint32_t*>(smem + S::kOffMisc + 12), ctl};
  const uint32_t tm_s = tmem + 4 * kN;  // two S^T buffers behind the output

  if (any && warp >= kLoadWarp) {
    // ------------------------------------------------------------ loaders
    const int grp = (warp - kLoadWarp) >> 2, tid = threadIdx.x - (kLoadWarp + 4 * grp) * 32;
    const int wrow = (tid >> 5) * 16 + (lane >> 3), piece = lane & 7;  // of the copies
    const int tok = (tid >> 5) * 16 + (lane & 15);  // the token that the lane looks up
    uint32_t kctr = 0;
    int t = seg.t0;
    bool have = !p.idle_producers;
    // moves to this group's next tile, n tiles on
    auto advance = [&](int n) {
      kctr += n;
      t += n;
      while (t >= seg.t1) {
        n = t - seg.t1;
        if (!next_seg<kSelected, kShared>(p, seg, feed)) {
          have = false;
          return;
        }
        t = seg.t0 + n;
      }
    };
    // A tile's tokens are looked up two steps ahead, positions and then page ids, one token a
    // lane; each value is used an iteration after its load was issued.
    bool whole1 = false, whole2 = false;  // every row sees all of the tile, which is one page
    int pos1 = 0, pos2 = 0;        // of the group's next tile, and of the one after it
    uint32_t rows1 = 0, rows2 = 0;  // rows of the unit that see the token, if its position is valid
    int32_t page1 = -1;
    const int32_t* table2 = a.page_table;
    auto positions = [&]() {  // of the walker's tile
      table2 = a.page_table + (int64_t)seg.u.seq * a.max_pages;
      pos2 = t * kTile + tok;
      rows2 = 0;
      if (kSelected) {
        if (pos2 < seg.u.min_len) {
          rows2 = 1;
          pos2 = a.idx[(int64_t)seg.u.r0 * a.k + pos2];
        }
        return;
      }
      whole2 = (t + 1) * kTile <= seg.u.min_len;
      if (whole2) {
        rows2 = (1u << seg.u.rows) - 1;
        return;
      }
#pragma unroll 4
      for (int r = 0; r < seg.u.rows; r++) {
        const int len = __shfl_sync(kFull, seg.u.len, r), end = __shfl_sync(kFull, seg.u.end, r), j = pos2 - len;
        const uint32_t word = j >= 0 && pos2 < end ? a.tree[(int64_t)(seg.u.r0 + r) * a.words + (j >> 5)] : 0;
        rows2 |= (uint32_t)(j < 0 || (word >> (j & 31) & 1)) << r;
      }
    };
    auto pages = [&]() {
      pos1 = pos2;
      whole1 = whole2;
      rows1 = pos2 >= 0 ? rows2 : 0;
      page1 = -1;
      if (rows1) {
        if (pos1 / kPage < a.max_pages) {
          page1 = table2[pos1 / kPage];
        } else {
          record_error(a.status, FP4IDX_ERR_BAD_LENGTH);
          rows1 = 0;
        }
      }
    };
    if (have && grp > 0) advance(grp);
    uint32_t kcur = kctr;
    bool have1 = have, tma = false;
    uint32_t last = 0;
    if (have) {
      positions();
      pages();
      advance(kStages);
      if (have) positions();
    }
    while (have1) {
      const int s = kcur % kStages;
      const uint32_t free = ((kcur / kStages) & 1) ^ 1;
      if (!mma::wait_warp(kempty(s, 0), free, ctl)) break;
      const bool in = (uint32_t)page1 < (uint32_t)a.num_pages;
      if (!in && rows1) record_error(a.status, FP4IDX_ERR_BAD_PAGE);
      const int slot = in ? page1 * kPage + (pos1 & (kPage - 1)) : -1;
      if (lane < 16) smem[S::kOffSeen + s * kTile + tok] = (uint8_t)(in ? rows1 : 0);
      const uint32_t dst = sb + s * S::kStageBytes;
      last = kcur;
      have1 = have;
      // (a page outside the cache takes the other path: its rows become zero)
      tma = !kSelected && __all_sync(kFull, whole1 && in);
      if (tma) {
        // a whole page: one box of 64 tokens x 64 dims a block, issued by the first warp
        const int row = __shfl_sync(kFull, page1, 0) * kPage;
        __syncwarp();
#pragma unroll
        for (int half = 0; half < 2; half++) {
          if (half && !mma::wait_warp(kempty(s, 1), free, ctl)) break;
          if (tid >= 32) {
            arrive_warp(kfull(s, half), lane);
          } else if (mma::elect_one()) {
            const int c0 = half ? 4 : 0, c1 = half ? kChunks : 4;
            ptx::mbar_arrive_expect_tx(kfull(s, half), (c1 - c0) * kTile * 128);
            for (int c = c0; c < c1; c++) mma::tma_2d(dst + c * (kTile * 128), &cache_map, c * 64, row, kfull(s, half));
          }
          __syncwarp();
        }
        kcur = kctr;
        if (have) {
          pages();
          advance(kStages);
          if (have) positions();
        }
        continue;
      }
      const uint16_t* src[4];
      uint32_t bytes[4];
#pragma unroll
      for (int g = 0; g < 4; g++) {
        const int of = __shfl_sync(kFull, slot, g * 4 + (lane >> 3));
        src[g] = a.cache + (int64_t)max(of, 0) * kWidth + piece * 8;
        bytes[g] = of >= 0 ? 16 : 0;
      }
#pragma unroll
      for (int c = 0; c < kChunks; c++) {
        if (c == 4) {
          mma::cp_async_commit();
          if (!mma::wait_warp(kempty(s, 1), free, ctl)) break;
        }
#pragma unroll
        for (int g = 0; g < 4; g++)
          mma::cp_async16(dst + c * (kTile * 128) + mma::sw128(wrow + g * 4, piece), src[g] + c * 64, bytes[g]);
      }
      mma::cp_async_commit();
      mma::cp_async_wait_group<1>();
      ptx::fence_proxy_async_smem();
      arrive_warp(kfull(s, 0), lane);
      kcur = kctr;
      if (have) {
        pages();
        advance(kStages);
        if (have) positions();
      }
      mma::cp_async_wait_group<0>();
      ptx::fence_proxy_async_smem();
      arrive_warp(kfull(s, 1), lane);
    }
    mma::cp_async_wait_all();
    // every copy lands before the CTA ends
    if (tma && tid < 32) {
      mma::wait_warp(kfull(last % kStages, 0), (last / kStages) & 1, ctl, false);
      mma::wait_warp(kfull(last % kStages, 1), (last / kStages) & 1, ctl, false);
    }
  } else if (any && warp == kQueryWarp) {
    // ------------------------------------------------------------ queries
    uint32_t ictr = 0;
    do {
      if (!mma::wait_warp(qempty, (ictr & 1) ^ 1, ctl)) break;
      ictr++;
      if (p.q_boxes) {
        // (columns behind the unit's get other rows' queries, or zeros behind the last row: what
        // comes of them is not stored)
        if (mma::elect_one()) {
          ptx::mbar_arrive_expect_tx(qfull, kChunks * S::kQChunk);
          const int row = seg.u.r0 * a.heads + seg.hb * p.hs;
#pragma unroll
          for (int c = 0; c < kChunks; c++) mma::tma_2d(sb + S::kOffQ + c * S::kQChunk, &q_map, c * 64, row, qfull);
        }
        __syncwarp();
        continue;
      }
      const int r0 = lane >> 3, pc = lane & 7;
      for (int col = r0; col < kN; col += 4) {
        const int r = col / p.hp, h = col % p.hp, head = seg.hb * p.hs + h;
        const bool in = r < seg.u.rows && h < p.hs && head < a.heads;
        const uint16_t* q = in ? a.q + ((int64_t)(seg.u.r0 + r) * a.heads + head) * kWidth + pc * 8 : a.q;
        const uint32_t dst = sb + S::kOffQ + mma::sw128(col, pc);
#pragma unroll
        for (int c = 0; c < kChunks; c++) mma::cp_async16(dst + c * S::kQChunk, q + (in ? c * 64 : 0), in ? 16 : 0);
      }
      mma::cp_async_wait_all();
      ptx::fence_proxy_async_smem();
      arrive_warp(qfull, lane);
    } while (next_seg<kSelected, kShared>(p, seg, feed, true));
    if (p.q_boxes && ictr > 0) mma::wait_warp(qfull, (ictr - 1) & 1, ctl, false);  // lands before the CTA ends
  } else if (any && warp == kAheadWarp) {
    // ------------------------------------------------------------ prefetches (two tokens a lane)
    uint32_t kctr = 0;
    volatile uint32_t* progress = reinterpret_cast<volatile uint32_t*>(smem + S::kOffMisc + 8);
    bool on = !p.idle_producers;
    do {
      for (int t = seg.t0; on && t < seg.t1; t++, kctr++) {
        if (kctr < kStages) continue;  // the loaders are at these already
        const int64_t t0 = clock64();
        while ((int32_t)(kctr - __shfl_sync(kFull, *progress, 0)) > (int32_t)kAhead) {
          __nanosleep(100);
          const int stop = *ctl.abort || clock64() - t0 > (int64_t)ctl.timeout_ns;  // only a hint: no error
          if (__shfl_sync(kFull, stop, 0)) {
            on = false;
            break;
          }
        }
#pragma unroll
        for (int g = 0; g < 2; g++) {
          int pos = t * kTile + lane + 32 * g;
          bool some = pos < (kSelected ? seg.u.min_len : seg.u.tiles * kTile) && seg.u.seq >= 0 && seg.u.seq < a.num_seqs;
          if (some && kSelected) pos = a.idx[(int64_t)seg.u.r0 * a.k + pos];
          if (some && pos >= 0 && pos / kPage < a.max_pages) {
            const int32_t page = a.page_table[(int64_t)seg.u.seq * a.max_pages + pos / kPage];
            if (page >= 0 && page < a.num_pages) {
              const uint8_t* row = reinterpret_cast<const uint8_t*>(a.cache + ((int64_t)page * kPage + pos % kPage) * kWidth);
#pragma unroll
              for (int c = 0; c < kWidth * 2; c += 128) pipe::prefetch_l2(row + c);
            }
          }
        }
      }
    } while (on && next_seg<kSelected, kShared>(p, seg, feed));
  } else if (any && warp == kScoreWarp) {
    // ------------------------------------------------------------ the first product (the warp as one)
    constexpr uint32_t kIdS = mma::idesc_bf16(64, kN, false, false);
    const uint32_t qd = mma::desc_lo(sb + S::kOffQ, 0), kd0 = mma::desc_lo(sb, 0);
    uint32_t stage = 0, phase = 0, buf = 0, q_phase = 0;
    bool ok = true;
    do {
      const uint32_t n = __shfl_sync(kFull, (uint32_t)(seg.t1 - seg.t0), 0);
      ok = mma::wait_warp(qfull, q_phase, ctl);
      q_phase ^= 1;
      for (uint32_t i = 0; ok && i < n; i++) {
        // The scores' buffer was last used two tiles ago.  Its reader is done once that
        // tile's second product has begun, which with two stages the loads wait for too.
        if (kStages > 2) {
          const uint32_t at = stage >= 2 ? stage - 2 : stage + kStages - 2;
          ok = mma::wait_warp(kempty(at, 0), (stage >= 2 ? phase : phase ^ 1), ctl);
          if (!ok) break;
        }
        const uint32_t kd = kd0 + stage * (S::kStageBytes >> 4), d = tm_s + buf * kN;
        ok = mma::wait_warp(kfull(stage, 0), phase, ctl);
        if (!ok) break;
        ptx::tc_fence_after();
        if (mma::elect_one()) {
#pragma unroll
          for (int c = 0; c < 4; c++)
#pragma unroll
            for (int e = 0; e < 4; e++)
              mma::mma_ss(d, kd + ((c * (kTile * 128) + e * 32) >> 4), qd + ((c * S::kQChunk + e * 32) >> 4), kIdS, (c | e) != 0);
        }
        __syncwarp();
        ok = mma::wait_warp(kfull(stage, 1), phase, ctl);
        if (!ok) break;
        if (mma::elect_one()) {
#pragma unroll
          for (int c = 4; c < kChunks; c++)
#pragma unroll
            for (int e = 0; e < 4; e++)
              mma::mma_ss(d, kd + ((c * (kTile * 128) + e * 32) >> 4), qd + ((c * S::kQChunk + e * 32) >> 4), kIdS, true);
          ptx::mma_commit(sfull(buf));
          if (i + 1 == n) ptx::mma_commit(qempty);
        }
        __syncwarp();
        buf ^= 1;
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
    } while (ok && next_seg<kSelected, kShared>(p, seg, feed));
    // nothing of this CTA's may be under way in the tensor cores when it ends
    if (mma::elect_one()) ptx::mma_commit(done);
    __syncwarp();
    mma::wait_warp(done, 0, ctl, false);
  } else if (any && warp == kOutWarp) {
    // ------------------------------------------------------------ the second product
    constexpr uint32_t kIdO = mma::idesc_bf16(128, kN, true, false);
    const uint32_t vd0 = mma::desc_lo(sb, kTile * 128);
    uint32_t stage = 0, tile = 0;
    bool ok = true;
    do {
      const uint32_t n = __shfl_sync(kFull, (uint32_t)(seg.t1 - seg.t0), 0);
      for (uint32_t i = 0; ok && i < n; i++, tile++) {
        ok = mma::wait_warp(pfull(tile & 1), (tile >> 1) & 1, ctl);
        if (!ok) break;
        ptx::tc_fence_after();
        const uint32_t vd = vd0 + stage * (S::kStageBytes >> 4), pd = mma::desc_lo(sb + S::off_p(stage), 0);
        if (mma::elect_one()) {
#pragma unroll
          for (int half = 0; half < 2; half++) {
#pragma unroll
            for (int ks = 0; ks < 4; ks++)
#pragma unroll
              for (int b = 2 * half; b < 2 * half + 2; b++)
                mma::mma_ss(tmem + b * kN, vd + ((b * (2 * kTile * 128) + ks * 2048) >> 4), pd + ((ks * 32) >> 4), kIdO,
                            ks > 0 || i > 0);
            ptx::mma_commit(kempty(stage, half));
          }
        }
        __syncwarp();
        if (++stage == kStages) stage = 0;
      }
    } while (ok && next_seg<kSelected, kShared>(p, seg, feed));
    if (mma::elect_one()) ptx::mma_commit(done);
    __syncwarp();
    mma::wait_warp(done, 0, ctl, false);
  } else if (any && warp < S::kSoftWarps) {
    // ------------------------------------------------------------ softmax and output
    const float cs = a.scale * 1.4426950408889634f;
    const int quad = lane & 3, r8 = lane >> 2;
    const int qw = warp & 3, col0 = (warp >> 2) * kMyCols;  // tensor-memory quarter, first column
    const uint32_t lanes = (uint32_t)(qw * 32) << 16;
    float* red = reinterpret_cast<float*>(smem + S::kOffRed);
    float* sm_m = reinterpret_cast<float*>(smem + S::kOffM);
    float* sm_f = reinterpret_cast<float*>(smem + S::kOffF);
    const int tok = qw * 16 + r8;  // and tok + 8
    uint32_t kctr = 0;
    bool ok = true, first_of_cta = true;
    do {
      const int n = seg.t1 - seg.t0;
      const uint32_t everyone = (1u << seg.u.rows) - 1;
      // of the thread's columns 8 j + 2 quad + {0, 1}; m starts low enough that any score raises it
      float2 m[kJ], l[kJ];
#pragma unroll
      for (int j = 0; j < kJ; j++) {
        m[j] = make_float2(kNoMax, kNoMax);
        l[j] = make_float2(0.f, 0.f);
      }
      for (int i = 0; i < n; i++, kctr++) {
        const int st = kctr % kStages;
        // a warp whose wait ran out goes on to the next vote, so that all four leave together
        ok = ok && mma::wait_warp(kfull(st, 0), (kctr / kStages) & 1, ctl);
        const uint32_t see0 = smem[S::kOffSeen + st * kTile + tok], see1 = smem[S::kOffSeen + st * kTile + tok + 8];
        const bool all_seen = __all_sync(kFull, (see0 & see1) == everyone);
        if (threadIdx.x == 0) *reinterpret_cast<volatile uint32_t*>(smem + S::kOffMisc + 8) = kctr;
        ok = ok && mma::wait_warp(sfull(kctr & 1), (kctr >> 1) & 1, ctl);
        ptx::tc_fence_after();
        // scores: v[2 j] of token tok, v[2 j + 1] of token tok + 8
        float2 v[2 * kJ];
        mma::ld_16x256b<kJ>(tm_s + (kctr & 1) * kN + col0 + lanes, reinterpret_cast<float*>(v));
        float mul = cs;
        bool zero0 = false, zero1 = false;
        if (!all_seen) {
          if (!kSelected && seg.u.rows > 1) {
            // A token that some rows see and others do not stays in the second product.  If
            // its value is not finite (then no score is), the value row is zeroed below and
            // the columns that see it get a NaN weight: NaN for those, nothing for the others.
#pragma unroll
            for (int half = 0; half < 2; half++) {
              const uint32_t see = half ? see1 : see0;
              bool odd = see != 0 && see != everyone;
#pragma unroll
              for (int j = 0; j < kJ; j++)
                odd = odd && !(fabsf(v[2 * j + half].x) < INFINITY) && !(fabsf(v[2 * j + half].y) < INFINITY);
              if (__any_sync(kFull, odd)) {
                bool bad = false;
                for (int c = quad; c < kValue / 8; c += 4) {
                  const uint4 u = *reinterpret_cast<const uint4*>(smem + st * S::kStageBytes + (c >> 3) * (kTile * 128) +
                                                                  mma::sw128(tok + 8 * half, c & 7));
                  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                  for (int e = 0; e < 4; e++)
                    bad = bad || (w[e] & 0x7F80u) == 0x7F80u || (w[e] & 0x7F800000u) == 0x7F800000u;
                }
                bad = (__ballot_sync(kFull, bad) >> (lane & 28) & 15u) != 0 && see != 0 && see != everyone;
                (half ? zero1 : zero0) = bad;
                if (bad) {
#pragma unroll
                  for (int j = 0; j < kJ; j++) v[2 * j + half] = make_float2(NAN, NAN);
                }
              }
            }
          }
#pragma unroll
          for (int j = 0; j < kJ; j++) {
            const int r = kSelected ? 0 : (col0 + 8 * j) / p.hp;
            const bool in0 = (see0 >> r) & 1, in1 = (see1 >> r) & 1;
            v[2 * j] = in0 ? make_float2(v[2 * j].x * cs, v[2 * j].y * cs) : make_float2(-INFINITY, -INFINITY);
            v[2 * j + 1] = in1 ? make_float2(v[2 * j + 1].x * cs, v[2 * j + 1].y * cs) : make_float2(-INFINITY, -INFINITY);
          }
          mul = 1.f;
        }
        // v[] becomes the exponents: scores, in powers of two, above the reference
        const float2 mul2 = make_float2(mul, mul);
        float most = -INFINITY;
        float2 x[2 * kJ];
#pragma unroll
        for (int j = 0; j < 2 * kJ; j++) {
          x[j] = mma::fma2(v[j], mul2, make_float2(-m[j >> 1].x, -m[j >> 1].y));
          most = fmaxf(most, fmaxf(x[j].x, x[j].y));
        }
        const bool raise = mma::bar_any(1, kSoft, most > kRaise || !ok);
        if (!kSelected && (zero0 || zero1)) {
          for (int c = quad; c < kValue / 8; c += 4) {
            uint8_t* row = smem + st * S::kStageBytes + (c >> 3) * (kTile * 128);
            if (zero0) *reinterpret_cast<uint4*>(row + mma::sw128(tok, c & 7)) = make_uint4(0, 0, 0, 0);
            if (zero1) *reinterpret_cast<uint4*>(row + mma::sw128(tok + 8, c & 7)) = make_uint4(0, 0, 0, 0);
          }
        }
        if (raise) {
          if (mma::bar_any(1, kSoft, !ok)) {
            ok = false;
            break;
          }
#pragma unroll
          for (int j = 0; j < kJ; j++) {
            float2 t = make_float2(fmaxf(v[2 * j].x * mul, v[2 * j + 1].x * mul), fmaxf(v[2 * j].y * mul, v[2 * j + 1].y * mul));
#pragma unroll
            for (int d = 4; d <= 16; d <<= 1) {
              t.x = fmaxf(t.x, __shfl_xor_sync(kFull, t.x, d));
              t.y = fmaxf(t.y, __shfl_xor_sync(kFull, t.y, d));
            }
            if (r8 == 0) *reinterpret_cast<float2*>(red + qw * kN + col0 + 8 * j + 2 * quad) = t;
          }
          ptx::named_bar_sync(1, kSoft);
#pragma unroll
          for (int j = 0; j < kJ; j++) {
            const int c = col0 + 8 * j + 2 * quad;
            float2 m1 = m[j];
#pragma unroll
            for (int q = 0; q < 4; q++) {
              const float2 t = *reinterpret_cast<const float2*>(red + q * kN + c);
              m1 = make_float2(fmaxf(m1.x, t.x), fmaxf(m1.y, t.y));
            }
            const float2 f = make_float2(m1.x == m[j].x ? 1.f : mma::exp2_approx(m[j].x - m1.x),
                                         m1.y == m[j].y ? 1.f : mma::exp2_approx(m[j].y - m1.y));
            if (qw == 0 && r8 == 0) *reinterpret_cast<float2*>(sm_f + c) = f;
            l[j] = make_float2(l[j].x * f.x, l[j].y * f.y);
            m[j] = m1;
            x[2 * j] = mma::fma2(v[2 * j], mul2, make_float2(-m1.x, -m1.y));
            x[2 * j + 1] = mma::fma2(v[2 * j + 1], mul2, make_float2(-m1.x, -m1.y));
          }
          ptx::named_bar_sync(1, kSoft);  // red is read, sm_f is written
        }
        uint32_t pk[2 * kJ];
#pragma unroll
        for (int j = 0; j < kJ; j++) {
          const float2 p0 = make_float2(mma::exp2_approx(x[2 * j].x), mma::exp2_approx(x[2 * j].y));
          const float2 p1 = make_float2(mma::exp2_approx(x[2 * j + 1].x), mma::exp2_approx(x[2 * j + 1].y));
          l[j] = mma::add2(l[j], mma::add2(p0, p1));
          pk[2 * j] = mma::pack_bf16(p0.x, p0.y);
          pk[2 * j + 1] = mma::pack_bf16(p1.x, p1.y);
        }
        if (raise && i > 0) {
          // the output is rescaled once the last tile's product is in it
          const uint32_t last = kctr - 1;
          ok = mma::wait_warp(kempty(last % kStages, 1), (last / kStages) & 1, ctl);
          if (!ok) continue;
          ptx::tc_fence_after();
#pragma unroll 1
          for (int b = 0; b < 4 * kMyCols; b += 16) {
            const int c = col0 + b % kMyCols, at = b / kMyCols * kN + c;
            float o[16];
            mma::ld_32x16(tmem + at + lanes, o);
#pragma unroll
            for (int e = 0; e < 16; e++) o[e] *= sm_f[c + e];
            mma::st_32x16(tmem + at + lanes, o);
          }
          ptx::tmem_wait_st();
        }
#pragma unroll
        for (int j = 0; j < kJ; j += 2) {
          const int col = col0 + 8 * (j + (lane >> 4)) + (lane & 7), tb = 2 * qw + ((lane >> 3) & 1);
          mma::stmatrix_x4_trans(sb + S::off_p(st) + mma::sw128(col, tb), pk[2 * j], pk[2 * j + 1], pk[2 * j + 2], pk[2 * j + 3]);
        }
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        arrive_warp(pfull(kctr & 1), lane);
      }
      if (mma::bar_any(1, kSoft, !ok)) break;
      // ---- the segment's output
      const bool begins = seg.t0 == 0, ends = seg.t1 == seg.u.tiles, whole = begins && ends;
#pragma unroll
      for (int j = 0; j < kJ; j++) {
#pragma unroll
        for (int d = 4; d <= 16; d <<= 1) {
          l[j].x += __shfl_xor_sync(kFull, l[j].x, d);
          l[j].y += __shfl_xor_sync(kFull, l[j].y, d);
        }
        const int c = col0 + 8 * j + 2 * quad;
        if (r8 == 0) *reinterpret_cast<float2*>(red + qw * kN + c) = l[j];
        if (r8 == 0 && qw == 0) *reinterpret_cast<float2*>(sm_m + c) = m[j];
      }
      ptx::named_bar_sync(1, kSoft);
      const int slot = 2 * blockIdx.x + (first_of_cta ? 0 : 1);
      first_of_cta = false;
      if (threadIdx.x < kN) {
        const int c = threadIdx.x;
        const float total = red[c] + red[kN + c] + red[2 * kN + c] + red[3 * kN + c];
        if (cluster > 1) {
          sm_f[c] = total;
        } else if (kShared || whole) {
          sm_f[c] = total == 0.f ? 0.f : 1.f / total;
          const int r = c / p.hp, h = c % p.hp, head = seg.hb * p.hs + h;
          if (a.lse && r < seg.u.rows && h < p.hs && head < a.heads)
            a.lse[(int64_t)(seg.u.r0 + r) * a.heads + head] =
                total == 0.f ? -INFINITY : (sm_m[c] + log2f(total)) * 0.6931471805599453f;
        } else {
          wk.ml[slot * 2 * kCols + c] = sm_m[c];
          wk.ml[slot * 2 * kCols + kCols + c] = total;
        }
      }
      if (!kShared && !whole && threadIdx.x == 0)
        wk.rec[slot] = Record{seg.u.r0, seg.u.rows, seg.hb, kUsed | (begins ? kBegins : 0) | (ends ? kEnds : 0)};
      const uint32_t last = kctr - 1;
      ok = mma::wait_warp(kempty(last % kStages, 1), (last / kStages) & 1, ctl);
      if (mma::bar_any(1, kSoft, !ok)) break;
      if (cluster > 1) break;  // the one piece: joined below
      ptx::tc_fence_after();
      // lane = dim, columns = heads: a warp writes 32 dims of one head at a time
      if (kShared || whole) {
#pragma unroll 1
        for (int r = 0; r < seg.u.rows; r++) {
          const int head0 = seg.hb * p.hs, heads = min(p.hs, a.heads - head0);
          uint16_t* dst = a.out + ((int64_t)(seg.u.r0 + r) * a.heads + head0) * kValue + qw * 32 + lane;
#pragma unroll 1
          for (int h = (warp >> 2) * 8; h < heads; h += 2 * S::kSoftWarps) {
            const int c = r * p.hp + h;
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; e++) f[e] = sm_f[c + e];
#pragma unroll
            for (int b = 0; b < 4; b++) {
              float o[8];
              mma::ld_32x8(tmem + b * kN + c + lanes, o);
#pragma unroll
              for (int e = 0; e < 8; e++)
                if (h + e < heads) dst[(h + e) * kValue + b * 128] = (uint16_t)mma::pack_bf16(o[e] * f[e], 0.f);
            }
          }
        }
      } else {
        float* dst = wk.o + (int64_t)slot * kCols * kValue + qw * 32 + lane;
#pragma unroll 1
        for (int c = col0; c < col0 + kMyCols; c += 8) {
#pragma unroll
          for (int b = 0; b < 4; b++) {
            float o[8];
            mma::ld_32x8(tmem + b * kN + c + lanes, o);
#pragma unroll
            for (int e = 0; e < 8; e++) dst[(c + e) * kValue + b * 128] = o[e];
          }
        }
      }
      ptx::tc_fence_before();
      ptx::named_bar_sync(1, kSoft);  // red, sm_m and sm_f are free again
    } while (next_seg<kSelected, kShared>(p, seg, feed));
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (cluster > 1) {
    // ---- the cluster's pieces are joined: each CTA for its share of the columns
    // All main loops are over, so shared memory is free: pieces of the CTA's columns at 0,
    // [piece][column][512] fp32, every piece's m and l in the query buffer.
    const int ctas = cluster, mine = blockIdx.x & (ctas - 1);  // two, four, eight or sixteen
    const int share = kN / ctas, shift = __ffs(share) - 1;
    float* gather = reinterpret_cast<float*>(smem + S::kOffQ);  // [piece][2][kN]
    float* sm_m = reinterpret_cast<float*>(smem + S::kOffM);
    float* sm_l = reinterpret_cast<float*>(smem + S::kOffF);
    mma::cluster_sync();
    for (int i = threadIdx.x; i < ctas * kN; i += S::kThreads) {
      const int c = i & (kN - 1), to = i / kN;
      mma::st_cluster(mma::map_shared(ptx::smem_addr(gather + (mine * 2) * kN + c), to), any ? sm_m[c] : kNoMax);
      mma::st_cluster(mma::map_shared(ptx::smem_addr(gather + (mine * 2 + 1) * kN + c), to), any ? sm_l[c] : 0.f);
    }
    // Every warp sends 32 dims of a column at a time, 128 adjacent bytes.  (Sixteen bytes a thread,
    // the columns of a dim together, take twice as long.)
    if (any) {
      const int qw = warp & 3;
      const uint32_t lanes = (uint32_t)(qw * 32) << 16, at = sb + (mine * share * kValue + qw * 32 + lane) * 4;
      float* local = reinterpret_cast<float*>(smem) + mine * share * kValue + qw * 32 + lane;
#pragma unroll 1
      for (int c = (warp >> 2) * 8; c < kN; c += S::kThreads / 128 * 8) {
#pragma unroll 1
        for (int b = 0; b < 4; b++) {
          float o[8];
          mma::ld_32x8(tmem + b * kN + c + lanes, o);
#pragma unroll
          for (int e = 0; e < 8; e++) {
            const int to = (c + e) >> shift, col = (c + e) & (share - 1);
            const int off = col * kValue + b * 128;
            if (to == mine) local[off] = o[e];
            else mma::st_cluster(mma::map_shared(at + off * 4, to), o[e]);
          }
        }
      }
    }
    mma::cluster_sync();
    for (int col = warp; col < share; col += S::kThreads / 32) {
      const int c = mine * share + col, r = c / p.hp, h = c % p.hp, head = seg.hb * p.hs + h;
      if (r >= seg.u.rows || h >= p.hs || head >= a.heads) continue;
      float top = kNoMax, total = 0.f, o[16] = {};
      for (int i = 0; i < ctas; i++) top = fmaxf(top, gather[(i * 2) * kN + c]);
      for (int i = 0; i < ctas; i++) {
        const float l = gather[(i * 2 + 1) * kN + c];
        if (l == 0.f) continue;  // no token, and nothing in the piece
        const float f = mma::exp2_approx(gather[(i * 2) * kN + c] - top);
        total += f * l;
        const float4* x = reinterpret_cast<const float4*>(smem) + ((i * share + col) * kValue) / 4 + lane;
#pragma unroll
        for (int q = 0; q < 4; q++) {
          const float4 y = x[32 * q];
          o[4 * q] += f * y.x;
          o[4 * q + 1] += f * y.y;
          o[4 * q + 2] += f * y.z;
          o[4 * q + 3] += f * y.w;
        }
      }
      const float inv = total == 0.f ? 0.f : 1.f / total;
      const int64_t row = (int64_t)(seg.u.r0 + r) * a.heads + head;
#pragma unroll
      for (int q = 0; q < 4; q++)
        *reinterpret_cast<uint2*>(a.out + row * kValue + q * 128 + lane * 4) =
            make_uint2(mma::pack_bf16(o[4 * q] * inv, o[4 * q + 1] * inv),
                       mma::pack_bf16(o[4 * q + 2] * inv, o[4 * q + 3] * inv));
      if (lane == 0 && a.lse) a.lse[row] = total == 0.f ? -INFINITY : (top + log2f(total)) * 0.6931471805599453f;
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
  }
  if (kShared && unit >= 0) {
    gave_up = *abort_flag;  // (the cluster's other CTAs count on this one until the end)
    if (threadIdx.x == 0) {
      for (int i = 0; i < S::kBars; i++) mma::mbar_inval(bar(i));
      init_barriers();
    }
    goto again;  // its barriers are seen behind the next __syncthreads
  }
  if (warp == kScoreWarp) ptx::tmem_dealloc(tmem, S::kTmemCols);
}

// ---------------------------------------------------------------- joining the pieces
// Block (u, y): the u-th unit that is in pieces, kBlockCols columns from kBlockCols * y on.  Its
// first piece is some CTA's last segment, the others are the first segments of the CTAs that
// follow.  A warp takes one column and every kGroups-th piece; the groups' sums are added in
// order.  Units have few pieces or many: one group of warps a column (all blocks are then
// resident at once), or 16.
template <int kBlockCols, int kGroups>
__global__ void __launch_bounds__(kBlockCols * kGroups * 32) combine_kernel(const Params p, int ctas) {
  __shared__ float sh_o[kGroups][kBlockCols][kGroups > 1 ? 128 : 1];
  __shared__ uint32_t sh_starts[kMaxCtas / 32], sh_ends[kMaxCtas / 32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const LatentArgs& a = p.a;
  const Work wk = work_view(a.workspace);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const auto starts = [](const Record& r) { return (r.flags & (kUsed | kBegins | kEnds)) == (kUsed | kBegins); };
  if (warp < kMaxCtas / 32) {
    const int c = threadIdx.x;
    bool first = false, last = false;
    if (c < ctas) {
      const Record r0 = wk.rec[2 * c], r1 = wk.rec[2 * c + 1];
      first = starts(r0) || starts(r1);
      last = (r0.flags & (kUsed | kBegins | kEnds)) == (kUsed | kEnds);
    }
    const uint32_t f = __ballot_sync(kFull, first), l = __ballot_sync(kFull, last);
    if (lane == 0) {
      sh_starts[warp] = f;
      sh_ends[warp] = l;
    }
  }
  __syncthreads();
  int c0 = -1, left = blockIdx.x;
#pragma unroll
  for (int w = 0; w < kMaxCtas / 32; w++) {
    const uint32_t f = sh_starts[w];
    const int n = __popc(f);
    if (c0 < 0 && left < n) c0 = 32 * w + __fns(f, 0, left + 1);
    left -= n;
  }
  if (c0 < 0) return;
  int c1 = ctas;
#pragma unroll
  for (int w = kMaxCtas / 32 - 1; w >= 0; w--) {
    uint32_t l = sh_ends[w];
    if (32 * w + 31 <= c0) l = 0;
    else if (32 * w <= c0) l &= ~0u << (c0 + 1 - 32 * w);
    if (l) c1 = 32 * w + __ffs(l) - 1;
  }
  if (c1 >= ctas) return;  // a run that gave up
  int slot0 = 2 * c0 + 1;
  Record rec = wk.rec[slot0];
  if (!starts(rec)) rec = wk.rec[--slot0];
  const int n = c1 - c0 + 1;
  const int grp = warp / kBlockCols, cl = warp % kBlockCols;
  const int col = blockIdx.y * kBlockCols + cl;
  const int r = col / p.hp, h = col % p.hp, head = rec.hb * p.hs + h;
  const bool in = r < rec.rows && h < p.hs && head < a.heads;
  auto slot_of = [&](int i) { return i == 0 ? slot0 : 2 * (c0 + i); };
  float top = -INFINITY, total = 0.f;
  float o[16] = {};
  if (in) {
    for (int i = lane; i < n; i += 32) top = fmaxf(top, wk.ml[slot_of(i) * 2 * kCols + col]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, d));
    for (int i = lane; i < n; i += 32) {
      const float* ml = wk.ml + slot_of(i) * 2 * kCols + col;
      total += mma::exp2_approx(ml[0] - top) * ml[kCols];
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(kFull, total, d);
#pragma unroll 2
    for (int i = grp; i < n; i += kGroups) {
      const int s = slot_of(i);
      const float f = mma::exp2_approx(wk.ml[s * 2 * kCols + col] - top);
      const float4* x = reinterpret_cast<const float4*>(wk.o + ((int64_t)s * kCols + col) * kValue) + lane;
#pragma unroll
      for (int q = 0; q < 4; q++) {
        const float4 y = x[32 * q];
        o[4 * q] += f * y.x;
        o[4 * q + 1] += f * y.y;
        o[4 * q + 2] += f * y.z;
        o[4 * q + 3] += f * y.w;
      }
    }
  }
  if constexpr (kGroups > 1) {
#pragma unroll
    for (int q = 0; q < 4; q++) {
      *reinterpret_cast<float4*>(&sh_o[grp][cl][lane * 4]) = make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
      __syncthreads();
      if (grp == 0) {
#pragma unroll
        for (int g = 1; g < kGroups; g++) {
          const float4 y = *reinterpret_cast<const float4*>(&sh_o[g][cl][lane * 4]);
          o[4 * q] += y.x;
          o[4 * q + 1] += y.y;
          o[4 * q + 2] += y.z;
          o[4 * q + 3] += y.w;
        }
      }
      __syncthreads();
    }
  }
  if (grp > 0 || !in) return;
  const float inv = total == 0.f ? 0.f : 1.f / total;
  const int64_t row = (int64_t)(rec.r0 + r) * a.heads + head;
#pragma unroll
  for (int q = 0; q < 4; q++)
    *reinterpret_cast<uint2*>(a.out + row * kValue + q * 128 + lane * 4) =
        make_uint2(mma::pack_bf16(o[4 * q] * inv, o[4 * q + 1] * inv),
                   mma::pack_bf16(o[4 * q + 2] * inv, o[4 * q + 3] * inv));
  if (lane == 0 && a.lse) a.lse[row] = total == 0.f ? -INFINITY : (top + log2f(total)) * 0.6931471805599453f;
}

// [rows, width] bf16, in boxes of box_rows rows x 64 dims, 128-byte swizzle.
bool encode_rows_of(CUtensorMap* map, const void* base, int64_t rows, int32_t width, int box_rows) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)width * 2};
  cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, es[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kWidth, int kN, bool kSelected>
cudaError_t launch(Params p, int ctas, bool may_split, cudaStream_t stream) {
  using S = Shape<kWidth, kN>;
  static_assert(S::kBytes <= 232448, "shared memory of a CTA");
  static_assert(S::kThreads <= kMaxWarps * 32, "");
  static_assert(kN * kValue * 4 <= S::kOffQ, "a cluster's pieces fit the stages");
  static_assert(sizeof(ScanShared) <= S::kChunks * S::kQChunk, "the scan's scratch fits the query buffer");
  const auto cut_kernel = latent_attn_kernel<kWidth, kN, kSelected, false>;
  const auto shared_kernel = latent_attn_kernel<kWidth, kN, kSelected, true>;
  // (a map that the kernel will not use is not encoded)
  CUtensorMap cache_map{}, q_map{};
  p.q_boxes = p.group == 1 || p.hp == p.a.heads;
  if ((!kSelected && !encode_rows_of(&cache_map, p.a.cache, (int64_t)p.a.num_pages * kPage, kWidth, kPage)) ||
      (p.q_boxes && !encode_rows_of(&q_map, p.a.q, (int64_t)p.a.n_rows * p.a.heads, kWidth, kN)))
    return cudaErrorInvalidValue;
  cudaError_t e = set_smem_attr_once(reinterpret_cast<const void*>(cut_kernel), S::kBytes);
  if (e == cudaSuccess) e = set_smem_attr_once(reinterpret_cast<const void*>(shared_kernel), S::kBytes);
  if (e != cudaSuccess) return e;
  // Both launches may begin while the one before them ends: each waits for it before its
  // first load or store (only prefetches into L2 come earlier).
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = stream;
  cfg.gridDim = dim3(ctas, 1, 1);
  cfg.blockDim = dim3(S::kThreads, 1, 1);
  cfg.dynamicSmemBytes = S::kBytes;
  // A cluster a unit, of the largest size of which the device holds that many, or a CTA a unit
  // (c = 1).  Units of several rows are counted as if every sequence's rows were adjacent; if
  // there are more, the clusters take them in rounds.
  const int runs = std::min(p.a.n_rows, p.a.num_seqs);
  const int units = p.group == 1 ? p.a.n_rows * p.hb : runs + (p.a.n_rows - runs) / p.group;
  const int tiles = ((kSelected ? p.a.k : p.a.max_context) + kTile - 1) / kTile;
  const bool one_chunk = p.group == 1 || p.a.n_rows <= S::kThreads;
  for (int c = 16; c >= 1 && one_chunk; c /= 2) {
    const int64_t share = (tiles + c - 1) / c, even = ((int64_t)tiles * units + ctas - 1) / ctas;
    if ((int64_t)units * c > ctas || share > even + kMore || (!kSelected && share > kMost)) continue;
    if (c > 1 && (c >= 2 * tiles || (c == 16 && tiles <= 8 * 3))) continue;  // as fast with half as many
    if (c > 1) {
      int fit = 0;
      e = resident_clusters(reinterpret_cast<const void*>(shared_kernel), c, S::kThreads, S::kBytes, &fit);
      if (e != cudaSuccess) return e;
      if (fit < units) continue;
      attr[1].id = cudaLaunchAttributeClusterDimension;
      attr[1].val.clusterDim.x = c;
      attr[1].val.clusterDim.y = 1;
      attr[1].val.clusterDim.z = 1;
      cfg.numAttrs = 2;
    }
    p.cluster = c;
    cfg.gridDim = dim3(units * c, 1, 1);
    return cudaLaunchKernelEx(&cfg, shared_kernel, cache_map, q_map, p);
  }
  if (p.whole) {
    e = cudaMemsetAsync(work_view(p.a.workspace).taken, 0, sizeof(uint32_t), stream);
    if (e != cudaSuccess) return e;
    cfg.numAttrs = 0;  // the launch before is not a kernel's
  }
  e = cudaLaunchKernelEx(&cfg, cut_kernel, cache_map, q_map, p);
  if (e != cudaSuccess || !may_split) return e;
  const int cut = std::min(ctas, p.a.n_rows * p.hb);  // units in pieces, at most
  const bool many = cut * 8 <= ctas;  // eight pieces a unit or more
  cfg.gridDim = dim3(cut, many ? kN / 2 : kN / 8, 1);
  cfg.blockDim = dim3(many ? 1024 : 256, 1, 1);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, many ? combine_kernel<2, 16> : combine_kernel<8, 1>, p, ctas);
}

template <bool kSelected>
cudaError_t launch_shape(const Params& p, int32_t width, int cols, int ctas, bool may_split, cudaStream_t stream) {
  if (width == 576) {
    if (cols <= 16) return launch<576, 16, kSelected>(p, ctas, may_split, stream);
    if (cols <= 32) return launch<576, 32, kSelected>(p, ctas, may_split, stream);
    return launch<576, 64, kSelected>(p, ctas, may_split, stream);
  }
  if (cols <= 16) return launch<512, 16, kSelected>(p, ctas, may_split, stream);
  if (cols <= 32) return launch<512, 32, kSelected>(p, ctas, may_split, stream);
  return launch<512, 64, kSelected>(p, ctas, may_split, stream);
}

}  // namespace

size_t latent_attn_workspace_bytes(int64_t, int32_t) { return kWorkBytes; }

cudaError_t launch_latent_attn(const LatentArgs& a, int32_t width, bool selected, cudaStream_t stream) {
  Params p{};
  p.a = a;
  p.hb = (a.heads + kCols - 1) / kCols;
  p.hs = (a.heads + p.hb - 1) / p.hb;
  p.hp = (p.hs + 7) / 8 * 8;
  p.group = 1;
  if (!selected) {
    // rows of one sequence share a pass when their columns fit; no more than a sequence has
    const int per_seq = (int)std::min<int64_t>(kMaxGroup, ((int64_t)a.n_rows + a.num_seqs - 1) / a.num_seqs);
    p.group = std::max(1, std::min(per_seq, kCols / p.hp));
  }
  p.wait_limit_ns = pipeline_wait_limit_ns();
  p.idle_producers = pipeline_idle_producers() ? 1 : 0;
  int sms = 0, dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int ctas = std::min(sms, kMaxCtas);
  const int units = a.n_rows * p.hb, rounds = (units + ctas - 1) / ctas, tiles = (a.k + kTile - 1) / kTile;
  p.whole = selected && units > ctas &&
            (units >= 2 * ctas || (int64_t)rounds * tiles <= (int64_t)tiles * units / ctas + kMore);
  const bool may_split = !p.whole && (selected ? a.k : a.max_context) > kTile;
  const int cols = p.group * p.hp;
  return selected ? launch_shape<true>(p, width, cols, ctas, may_split, stream)
                  : launch_shape<false>(p, width, cols, ctas, may_split, stream);
}

}  // namespace fp4idx
