// Expanded latent attention on the tensor cores: causal attention over packed prompts,
// per-head keys (128 own dims and 64 rotated ones that the heads share) and values (128 dims).
//
// A CTA takes 256 consecutive query rows of one (sequence, head), as two tiles of 128 that
// share the key and value tiles (112 tokens) in shared memory:
//   S = Q K^T          M = 128 rows, N = 112 tokens, K = 192     (Q, K in shared memory)
//   P = exp2(c S - m)  in place of S in tensor memory, bf16
//   O += P V           M = 128 rows, N = 128 dims, K = 112       (P in tensor memory)
// Each tile has a warp that issues its products in bursts (PV, then S of the next tokens); the
// warps take turns, so that one tile's softmax, and the few hundred cycles from a barrier to
// the next issue, pass while the other's burst runs.  (Without turns their MMAs interleave,
// both tiles' scores are done at once, and the tensor cores then wait for both softmaxes:
// 1.06 ms instead of 0.85 for prompts of 6,000 and 4,000 tokens with 64 heads.)
// Bound by the tensor cores and the shared memory that feeds them: a step of 112 tokens takes
// 2,900 cycles, its MMAs alone (two tiles, measured apart) 2,400; 1.34 PFLOP/s over those
// prompts (795 us with changing inputs among other work, 750 us repeated by themselves), of which
// 2,560 CTAs' set-up and output cost a seventh.
//   warps 0-7, 8-15 softmax and output of tile 0, 1: two threads a row, 56 columns each
//   warps 16, 17    issue the MMAs of tile 0, 1
//   warp 18         issues the TMA loads into a ring of nine 14 KB blocks (112 tokens x 64
//                   dims): three a key tile, two a value tile.  Tiles of 128 tokens leave
//                   room for eight: two of a step's five blocks then come when they are
//                   needed, not before (800 us)
// m is raised only when the weights of a row's half tile sum to more than 2^16, so O is hardly
// ever rescaled and no maximum is taken after the first tile; the result depends on m by rounding only.
// Queries of longer contexts have smaller block indices: the longest work starts first.
//
// Where all blocks together are few, a cluster of two, four or eight CTAs takes a block, each a
// share of its key tiles, and joins O, m and l through distributed shared memory: each CTA sends
// its weighted O of every row to the CTA that adds that row up.
#include <algorithm>
#include <type_traits>

#include "latent.cuh"
#include "mma_bf16.cuh"

namespace fp4idx {
namespace {

using pipe::Ctl;
using pipe::kFull;

constexpr int kKey = FP4IDX_PREFILL_KEY, kVal = FP4IDX_PREFILL_VALUE;
constexpr int kRows = 128, kTokens = 112, kHalf = kTokens / 2;
constexpr int kMmaWarp = 16, kLoadWarp = 18, kThreads = 608;
constexpr int kRing = 9;
constexpr uint32_t kQBlock = kRows * 128, kBlock = kTokens * 128;  // bytes: rows of 64 bf16
constexpr uint32_t kOffRing = 6 * kQBlock;  // behind the two query tiles
constexpr uint32_t kOffBar = kOffRing + kRing * kBlock;
// full[9], empty[9], qfull[2], sfull[2], pfull[2], ofull[2], done, tail, issued[2]
constexpr int kBars = 2 * kRing + 12;
constexpr uint32_t kOffMisc = kOffBar + kBars * 8;
constexpr uint32_t kOffRed = kOffMisc + 16;  // [tile][half][row] floats
constexpr uint32_t kOffMl = kOffRed + 4 * kRows * 4;  // [m, l][row of both tiles] floats
constexpr uint32_t kBytes = kOffMl + 4 * kRows * 4;
constexpr int kMaxCluster = 8;
constexpr uint32_t kOffParts = kMaxCluster * 4 * kRows * 4;  // of the join: behind every CTA's m and l
static_assert(kOffParts + 2 * kRows * kVal * 4 <= kOffBar, "a cluster's pieces fit the tiles");
static_assert(kBytes <= 232448, "shared memory of a CTA");
constexpr uint32_t kTmO = 256;  // tensor memory: S0, S1 at 0 and 128, O0, O1 behind them
constexpr float kRaise = 65536.f, kNoMax = -3.0e38f;

struct Params {
  PrefillArgs a;
  uint64_t wait_limit_ns;
  int32_t idle_producers;
  int32_t cluster;  // CTAs that share a block's keys
};

__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
// kSplit: a cluster a block (a kernel of its own: with both in one, prompts took 2 to 4 % longer).
template <bool kSplit>
__global__ void __launch_bounds__(kThreads, 1) latent_prefill_kernel(const __grid_constant__ CUtensorMap q_map,
                                                                    const __grid_constant__ CUtensorMap kv_map,
                                                                    const __grid_constant__ CUtensorMap r_map,
                                                                    const __grid_constant__ Params p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const PrefillArgs& a = p.a;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int seq = blockIdx.z, head = blockIdx.y;
  const int64_t q0 = a.cu_q[seq], q1 = a.cu_q[seq + 1], k1 = a.cu_kv[seq + 1];
  int64_t k0 = a.cu_kv[seq];
  if (q0 < 0 || q1 < q0 || q1 > a.n_q || k0 < 0 || k1 < k0 || k1 > a.n_kv || q1 - q0 > a.max_q || k1 - k0 > a.max_kv) {
    if (threadIdx.x == 0) record_error(a.status, FP4IDX_ERR_BAD_LENGTH);
    return;
  }
  const int nq = (int)(q1 - q0), all = (int)(k1 - k0);
  const int ctas = kSplit ? p.cluster : 1, rank = blockIdx.x & (ctas - 1);
  const int i0 = (int)((gridDim.x - 1 - blockIdx.x) >> (__ffs(ctas) - 1)) * 2 * kRows;
  if (i0 >= nq) return;
  // key tiles of the two query tiles: row i sees the keys before all - nq + i + 1
  int tiles[2];
#pragma unroll
  for (int t = 0; t < 2; t++) {
    const int last = min(nq, i0 + (t + 1) * kRows);  // rows before this one
    const int see = min(all, all - nq + last);
    tiles[t] = i0 + t * kRows < nq && see > 0 ? (see + kTokens - 1) / kTokens : 0;
  }
  // the CTA's share of them; from here on keys count from its first, of which nk lie before its end
  int nk = all, before = all - nq;  // row i sees before + i + 1
  if (kSplit) {
    const int total = max(tiles[0], tiles[1]), j0 = total * rank / ctas, j1 = total * (rank + 1) / ctas;
#pragma unroll
    for (int t = 0; t < 2; t++) tiles[t] = max(j0, min(j1, tiles[t])) - j0;
    nk = min(all, j1 * kTokens) - j0 * kTokens;
    before -= j0 * kTokens;
    k0 += j0 * kTokens;
  }
  const int n0 = tiles[0], n1 = tiles[1], n = max(n0, n1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t sb = ptx::smem_addr(smem);
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(smem + kOffMisc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffMisc + 4);
  const auto bar = [&](int i) { return sb + kOffBar + i * 8; };
  const auto full = [&](int i) { return bar(i); };
  const auto empty = [&](int i) { return bar(kRing + i); };
  const auto qfull = [&](int t) { return bar(2 * kRing + t); };
  const auto sfull = [&](int t) { return bar(2 * kRing + 2 + t); };
  const auto pfull = [&](int t) { return bar(2 * kRing + 4 + t); };
  const auto ofull = [&](int t) { return bar(2 * kRing + 6 + t); };
  const uint32_t done = bar(2 * kRing + 8), tail = bar(2 * kRing + 9);
  const auto issued = [&](int t) { return bar(2 * kRing + 10 + t); };
  // The loading warp sets the barriers up, so that its first loads need not wait for the others.
  const auto load = [&](int b) {  // block b of the stream, by one thread
    const int s = b % kRing, j = b / 5, c = b % 5, row = (int)k0 + j * kTokens;
    const uint32_t dst = sb + kOffRing + s * kBlock;
    ptx::mbar_arrive_expect_tx(full(s), kBlock);
    if (c == 2) mma::tma_2d(dst, &r_map, 0, row, full(s));
    else tma_3d(dst, &kv_map, c < 2 ? c * 64 : (c - 1) * 64, head, row, full(s));
  };
  // block b of the stream: key tile j is blocks 5 j .. 5 j + 2, value tile j 5 j + 3, 5 j + 4
  const int blocks = p.idle_producers ? 0 : 5 * n, early = min(blocks, kRing);
  if (warp == kLoadWarp && mma::elect_one()) {
    for (int i = 0; i < kRing; i++) {
      ptx::mbar_init(full(i), 1);
      ptx::mbar_init(empty(i), 2);  // both tiles
    }
    for (int t = 0; t < 2; t++) {
      ptx::mbar_init(qfull(t), 1);
      ptx::mbar_init(sfull(t), 1);
      ptx::mbar_init(pfull(t), 8);
      ptx::mbar_init(ofull(t), 1);
      ptx::mbar_init(issued(t), 1);
    }
    ptx::mbar_init(done, 2);
    ptx::mbar_init(tail, 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
    ptx::fence_proxy_async_smem();
    for (int t = 0; t < 2; t++) {
      if (tiles[t] == 0 || p.idle_producers) continue;
      ptx::mbar_arrive_expect_tx(qfull(t), 3 * kQBlock);
      for (int c = 0; c < 3; c++)
        tma_3d(sb + (3 * t + c) * kQBlock, &q_map, c * 64, head, (int)q0 + i0 + t * kRows, qfull(t));
      if (t == 0)
        for (int b = 0; b < min(early, 3); b++) load(b);
    }
    for (int b = tiles[0] && !p.idle_producers ? min(early, 3) : 0; b < early; b++) load(b);
  }
  if (warp == kMmaWarp) ptx::tmem_alloc(ptx::smem_addr(tmem_slot), 512);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Ctl ctl{abort_flag, a.status, 2 * p.wait_limit_ns};  // in cycles

  if (warp == kLoadWarp) {
    // ------------------------------------------------------------ loads
    bool ok = true;
    int b = early;
    for (; b < blocks; b++) {
      ok = mma::wait_warp(empty(b % kRing), ((b / kRing) & 1) ^ 1, ctl);
      if (!ok) break;
      if (mma::elect_one()) load(b);
      __syncwarp();
    }
    // A value tile that ends behind the sequence: its rows there (another sequence's, or
    // anything) become zero, since a weight of zero does not hide a NaN.
    const int rows = nk - (n - 1) * kTokens;
    if (ok && blocks > 0 && rows < kTokens) {
      for (int x = blocks - 2; x < blocks; x++) {
        ok = ok && mma::wait_warp(full(x % kRing), (x / kRing) & 1, ctl);
        if (!ok) break;
        uint8_t* v = smem + kOffRing + (x % kRing) * kBlock;
        for (int i = rows * 8 + lane; i < kTokens * 8; i += 32) *reinterpret_cast<uint4*>(v + i * 16) = make_uint4(0, 0, 0, 0);
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (ok && lane == 0) ptx::mbar_arrive(tail);
    }
    // every copy lands before the CTA ends
    for (int x = max(0, b - kRing); x < b; x++) mma::wait_warp(full(x % kRing), (x / kRing) & 1, ctl, false);
    if (!p.idle_producers) {
      for (int t = 0; t < 2; t++)
        if (tiles[t] > 0) mma::wait_warp(qfull(t), 0, ctl, false);
    }
  } else if (warp >= kMmaWarp) {
    // ------------------------------------------------------------ MMA issue (the warp as one)
    constexpr uint32_t kIdS = mma::idesc_bf16(128, kTokens, false, false);
    constexpr uint32_t kIdO = mma::idesc_bf16(128, 64, false, true);
    const int t = __shfl_sync(kFull, warp - kMmaWarp, 0), nt = t ? n1 : n0;
    const uint32_t qd = mma::desc_lo(sb + t * 3 * kQBlock, 0), kd = mma::desc_lo(sb + kOffRing, 0);
    const uint32_t vd = mma::desc_lo(sb + kOffRing, kBlock);
    const uint32_t ts = tmem + t * 128, to = tmem + kTmO + t * 128;
    uint32_t slot = 0, phase = 0;  // of the stream's next block
    const auto next = [&]() {
      if (++slot == kRing) {
        slot = 0;
        phase ^= 1;
      }
    };
    bool ok = nt == 0 || mma::wait_warp(qfull(t), 0, ctl);
    // the stream in order: keys 0, [values j, keys j + 1] ...; the value tile's two blocks may lie
    // on either side of the ring's end, so each has its own products (64 dims)
    uint32_t k_slot[3], k_phase[3];
    const auto keys = [&]() {
#pragma unroll
      for (int c = 0; c < 3; c++) {
        k_slot[c] = slot;
        k_phase[c] = phase;
        next();
      }
    };
    const auto wait_keys = [&]() {
#pragma unroll
      for (int c = 0; c < 3; c++) ok = ok && mma::wait_warp(full(k_slot[c]), k_phase[c], ctl);
    };
    const auto scores = [&]() {  // by the elected thread
#pragma unroll
      for (int c = 0; c < 3; c++) {
        const uint32_t kb = kd + k_slot[c] * (kBlock >> 4);
#pragma unroll
        for (int e = 0; e < 4; e++)
          mma::mma_ss(ts, qd + ((c * kQBlock + e * 32) >> 4), kb + ((e * 32) >> 4), kIdS, (c | e) != 0);
        ptx::mma_commit(empty(k_slot[c]));
      }
      ptx::mma_commit(sfull(t));
    };
    // burst k of a tile is PV of tile k - 1 and S of tile k; order: (0, tile 0), (0, tile 1), (1, tile 0) ...
    const int others = t ? n0 : n1;
    const auto wait_turn = [&](int k) {
      const int before = t ? k : k - 1;  // the other tile's burst before this one
      if (ok && others > 0 && before >= 0 && before <= others) ok = mma::wait_warp(issued(t ^ 1), before & 1, ctl);
    };
    if (nt > 0) {
      keys();
      wait_keys();
      wait_turn(0);
      if (ok) {
        ptx::tc_fence_after();
        if (mma::elect_one()) scores();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(issued(t));
      }
    }
    for (int j = 0; ok && j < nt; j++) {
      const uint32_t v_slot[2] = {slot, slot + 1 == kRing ? 0 : slot + 1};
      const uint32_t v_phase[2] = {phase, slot + 1 == kRing ? phase ^ 1 : phase};
      next();
      next();
      if (j + 1 < n) keys();
      ok = mma::wait_warp(full(v_slot[0]), v_phase[0], ctl) && mma::wait_warp(full(v_slot[1]), v_phase[1], ctl);
      if (ok && nk < (j + 1) * kTokens) ok = mma::wait_warp(tail, 0, ctl);
      if (j + 1 < nt) wait_keys();
      ok = ok && mma::wait_warp(pfull(t), j & 1, ctl);
      wait_turn(j + 1);
      if (!ok) break;
      ptx::tc_fence_after();
      const uint32_t vb0 = vd + v_slot[0] * (kBlock >> 4), vb1 = vd + v_slot[1] * (kBlock >> 4);
      if (mma::elect_one()) {
#pragma unroll
        for (int e = 0; e < kTokens / 16; e++) mma::mma_ts(to, ts + e * 8, vb0 + ((e * 2048) >> 4), kIdO, j > 0 || e > 0);
        ptx::mma_commit(empty(v_slot[0]));
#pragma unroll
        for (int e = 0; e < kTokens / 16; e++) mma::mma_ts(to + 64, ts + e * 8, vb1 + ((e * 2048) >> 4), kIdO, j > 0 || e > 0);
        ptx::mma_commit(empty(v_slot[1]));
        if (j + 1 == nt) ptx::mma_commit(ofull(t));
        else scores();
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(issued(t));
    }
    // blocks that only the other tile uses: given back as they come
    if (ok && nt < n) {
      if (nt == 0) keys();
      for (int j = nt; ok && j < n; j++) {
        if (j > nt) keys();
        for (int c = 0; ok && c < 5; c++) {
          const uint32_t sl = c < 3 ? k_slot[c] : slot, ph = c < 3 ? k_phase[c] : phase;
          if (c >= 3) next();
          ok = mma::wait_warp(full(sl), ph, ctl);
          if (ok && lane == 0) ptx::mbar_arrive(empty(sl));
        }
      }
    }
    if (mma::elect_one()) ptx::mma_commit(done);
    __syncwarp();
    mma::wait_warp(done, 0, ctl, false);
  } else {
    // ------------------------------------------------------------ softmax and output
    const int t = warp >> 3, half = (warp >> 2) & 1, qw = warp & 3, row = qw * 32 + lane;
    const int i = i0 + t * kRows + row;  // the thread's query row in its sequence
    const int nt = t ? n1 : n0;
    const int pair = 1 + t * 4 + qw;  // named barrier of the two warps that share rows
    const uint32_t lanes = (uint32_t)(qw * 32) << 16;
    const uint32_t ts = tmem + t * 128 + lanes, to = tmem + kTmO + t * 128 + half * 64 + lanes;
    float* red = reinterpret_cast<float*>(smem + kOffRed) + t * 2 * kRows + row;
    const float cs = a.scale * 1.4426950408889634f;
    const float2 cs2 = make_float2(cs, cs);
    const int limit = min(nk, before + i + 1);       // keys before this one are seen
    const int least = before + i0 + t * kRows + 1;   // ... by the tile's first row
    float m = kNoMax, l = 0.f;
    bool ok = true;
    for (int j = 0; j < nt; j++) {
      // a warp whose wait ran out goes on to the next vote, so that the pair leaves together
      ok = ok && mma::wait_warp(sfull(t), j & 1, ctl);
      ptx::tc_fence_after();
      const int seen = limit - j * kTokens - half * kHalf;  // columns before this one are seen
      const bool masked = min(least, nk) < (j + 1) * kTokens;
      uint32_t pk[kHalf / 2];
      float sum;
      const auto weights = [&](auto mask) {  // mask: whether some columns are not seen
        float2 v[kHalf / 2];
        mma::ld_32x56(ts + half * kHalf, reinterpret_cast<float*>(v));
        const float2 nm = make_float2(-m, -m);
        float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int e = 0; e < kHalf / 2; e++) {
          float2 x = mma::fma2(v[e], cs2, nm);
          if (decltype(mask)::value) {
            if (2 * e >= seen) x.x = -INFINITY;
            if (2 * e + 1 >= seen) x.y = -INFINITY;
          }
          const float2 w = make_float2(mma::exp2_approx(x.x), mma::exp2_approx(x.y));
          acc[e & 1] = mma::add2(acc[e & 1], w);
          pk[e] = mma::pack_bf16(w.x, w.y);
        }
        sum = (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
      };
      const auto all_weights = [&]() {
        if (masked) weights(std::true_type{});
        else weights(std::false_type{});
      };
      if (j > 0) all_weights();
      if (mma::bar_any(pair, 64, j == 0 || sum > kRaise || !ok)) {
        if (mma::bar_any(pair, 64, !ok)) {
          ok = false;
          break;
        }
        // the scores are still there: no weight is stored before both warps have voted
        float top = -INFINITY;
        {
          float v[kHalf];
          mma::ld_32x56(ts + half * kHalf, v);
#pragma unroll
          for (int e = 0; e < kHalf; e++)
            if (!masked || e < seen) top = fmaxf(top, v[e] * cs);
        }
        red[half * kRows] = top;
        ptx::named_bar_sync(pair, 64);
        const float m1 = fmaxf(m, fmaxf(red[0], red[kRows]));
        if (j > 0) {
          // the scores' commit came after the last tile's product into O
          const float f = m1 == m ? 1.f : mma::exp2_approx(m - m1);
          l *= f;
#pragma unroll 1
          for (int c = 0; c < 64; c += 16) {
            float o[16];
            mma::ld_32x16(to + c, o);
#pragma unroll
            for (int e = 0; e < 16; e++) o[e] *= f;
            mma::st_32x16(to + c, o);
          }
          ptx::tmem_wait_st();
        }
        m = m1;
        all_weights();
        ptx::named_bar_sync(pair, 64);  // red is read
      }
      l += sum;
      mma::st_32x28(ts + half * (kHalf / 2), pk);
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(pfull(t));
    }
    ok = ok && (nt == 0 || mma::wait_warp(ofull(t), 0, ctl));
    const bool fine = !mma::bar_any(pair, 64, !ok);
    if (fine) {
      red[half * kRows] = l;
      ptx::named_bar_sync(pair, 64);
      l = red[0] + red[kRows];
    }
    if (kSplit) {
      float* ml = reinterpret_cast<float*>(smem + kOffMl) + t * kRows + row;
      if (half == 0) {
        ml[0] = fine ? m : kNoMax;
        ml[2 * kRows] = fine ? l : 0.f;
      }
    } else if (fine) {
      const float inv = l == 0.f ? 0.f : 1.f / l;
      // through the tile's query blocks, which are free: a warp's 32 rows of 128 bytes
      uint8_t* st = smem + t * 3 * kQBlock + (warp & 7) * 4096;
      if (nt > 0) {
        ptx::tc_fence_after();
#pragma unroll
        for (int c = 0; c < 2; c++) {
          float o[32];
          mma::ld_32x32(to + c * 32, o);
#pragma unroll
          for (int e = 0; e < 4; e++) {
            const float* x = o + 8 * e;
            const uint4 u = make_uint4(mma::pack_bf16(x[0] * inv, x[1] * inv), mma::pack_bf16(x[2] * inv, x[3] * inv),
                                       mma::pack_bf16(x[4] * inv, x[5] * inv), mma::pack_bf16(x[6] * inv, x[7] * inv));
            *reinterpret_cast<uint4*>(st + mma::sw128(lane, c * 4 + e)) = u;
          }
        }
      }
      __syncwarp();
      const int64_t r0 = q0 + i0 + t * kRows + qw * 32;
      const int rows = min(32, nq - (i0 + t * kRows + qw * 32));
      for (int r = lane >> 3; r < rows; r += 4) {
        const int pc = lane & 7;
        const uint4 u = nt > 0 ? *reinterpret_cast<const uint4*>(st + mma::sw128(r, pc)) : make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4*>(a.out + ((r0 + r) * a.heads + head) * kVal + half * 64 + pc * 8) = u;
      }
      if (i < nq && half == 0 && a.lse)
        a.lse[(q0 + i) * a.heads + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (kSplit) {
    // ---- the cluster's pieces are joined, a share of the rows by each CTA; all of shared memory
    // before the barriers is free
    const int share = 2 * kRows / ctas, shift = __ffs(share) - 1;
    float* gather = reinterpret_cast<float*>(smem);  // [CTA][m, l][row]
    const float* ml = reinterpret_cast<const float*>(smem + kOffMl);
    mma::cluster_sync();
    for (int x = threadIdx.x; x < ctas * 4 * kRows; x += kThreads) {
      const int at = x & (4 * kRows - 1);
      mma::st_cluster(mma::map_shared(ptx::smem_addr(gather + rank * 4 * kRows + at), x / (4 * kRows)), ml[at]);
    }
    mma::cluster_sync();
    const auto weigh = [&](int r, float& top, float& sum) {  // of row r of the block
      top = kNoMax;
      sum = 0.f;
      for (int c = 0; c < ctas; c++) top = fmaxf(top, gather[c * 4 * kRows + r]);
      for (int c = 0; c < ctas; c++) {
        const float l = gather[(c * 4 + 2) * kRows + r];
        if (l != 0.f) sum += l * mma::exp2_approx(gather[c * 4 * kRows + r] - top);
      }
    };
    float* parts = reinterpret_cast<float*>(smem + kOffParts);  // [CTA][dim][row of the share]
    if (warp < kMmaWarp) {
      const int t = warp >> 3, half = (warp >> 2) & 1, qw = warp & 3, r = t * kRows + qw * 32 + lane;
      float top, sum;
      weigh(r, top, sum);
      const float f = mma::exp2_approx(ml[r] - top) / sum;
      const bool some = i0 + r < nq && ml[2 * kRows + r] != 0.f;
      if (__any_sync(kFull, some)) {
        const uint32_t at = mma::map_shared(
            ptx::smem_addr(parts + (rank * kVal + half * 64) * share + (r & (share - 1))), r >> shift);
#pragma unroll
        for (int c = 0; c < 64; c += 16) {
          float o[16];
          mma::ld_32x16(tmem + kTmO + t * 128 + half * 64 + c + ((uint32_t)(qw * 32) << 16), o);
          if (some) {
#pragma unroll
            for (int e = 0; e < 16; e++) mma::st_cluster(at + (c + e) * share * 4, o[e] * f);
          }
        }
      }
    }
    mma::cluster_sync();
    for (int x = threadIdx.x; x < share * (kVal / 8); x += kThreads) {
      const int lr = x & (share - 1), d = (x >> shift) * 8, r = rank * share + lr;
      if (i0 + r >= nq) continue;
      float o[8] = {};
      for (int c = 0; c < ctas; c++) {
        if (gather[(c * 4 + 2) * kRows + r] == 0.f) continue;  // nothing seen there, nothing sent
#pragma unroll
        for (int e = 0; e < 8; e++) o[e] += parts[(c * kVal + d + e) * share + lr];
      }
      const int64_t out = (q0 + i0 + r) * a.heads + head;
      *reinterpret_cast<uint4*>(a.out + out * kVal + d) =
          make_uint4(mma::pack_bf16(o[0], o[1]), mma::pack_bf16(o[2], o[3]), mma::pack_bf16(o[4], o[5]), mma::pack_bf16(o[6], o[7]));
      if (d == 0 && a.lse) {
        float top, sum;
        weigh(r, top, sum);
        a.lse[out] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
      }
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
  }
  if (warp == kMmaWarp) ptx::tmem_dealloc(tmem, 512);
}

// [rows, heads, width] bf16, in boxes of box_rows rows of one head x 64 dims, 128-byte swizzle.
bool encode_heads(CUtensorMap* map, const void* base, int64_t rows, int32_t heads, int32_t width, int box_rows) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)rows};
  cuuint64_t strides[2] = {(cuuint64_t)width * 2, (cuuint64_t)width * 2 * heads};
  cuuint32_t box[3] = {64, 1, (cuuint32_t)box_rows}, es[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool encode_rope(CUtensorMap* map, const void* base, int64_t rows) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {64, (cuuint64_t)rows};
  cuuint64_t strides[1] = {128};
  cuuint32_t box[2] = {64, kTokens}, es[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t launch_latent_prefill(const PrefillArgs& a, cudaStream_t stream) {
  Params p{a, pipeline_wait_limit_ns(), pipeline_idle_producers() ? 1 : 0, 1};
  CUtensorMap q_map, kv_map, r_map;
  // without any key the maps are never used: they then describe the queries' memory
  const bool keys = a.n_kv > 0;
  if (!encode_heads(&q_map, a.q, a.n_q, a.heads, kKey, kRows) ||
      !encode_heads(&kv_map, keys ? a.kv : a.q, keys ? a.n_kv : 1, keys ? a.heads : 1, keys ? 256 : 64, kTokens) ||
      !encode_rope(&r_map, keys ? a.k_rope : a.q, keys ? a.n_kv : 1))
    return cudaErrorInvalidValue;
  const void* split = reinterpret_cast<const void*>(latent_prefill_kernel<true>);
  cudaError_t e = set_smem_attr_once(reinterpret_cast<const void*>(latent_prefill_kernel<false>), kBytes);
  if (e == cudaSuccess) e = set_smem_attr_once(split, kBytes);
  if (e != cudaSuccess) return e;
  dim3 grid((a.max_q + 2 * kRows - 1) / (2 * kRows), a.heads, a.n_seqs);
  // A cluster a block where they all fit at once and a CTA keeps two key tiles or more.
  const int64_t blocks = (int64_t)grid.x * grid.y * grid.z;
  const int tiles = (int)(((int64_t)a.max_kv + kTokens - 1) / kTokens);
  for (int c = kMaxCluster; c >= 2; c /= 2) {
    if (tiles < 2 * c) continue;
    int fit = 0;
    e = resident_clusters(split, c, kThreads, kBytes, &fit);
    if (e != cudaSuccess) return e;
    if (fit < blocks) continue;
    p.cluster = c;
    grid.x *= c;
    return launch_early(latent_prefill_kernel<true>, grid, kThreads, kBytes, c, stream, q_map, kv_map, r_map, p);
  }
  return launch_early(latent_prefill_kernel<false>, grid, kThreads, kBytes, 1, stream, q_map, kv_map, r_map, p);
}

}  // namespace fp4idx
