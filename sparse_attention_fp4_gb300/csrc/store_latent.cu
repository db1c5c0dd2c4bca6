// Latent store: RMSNorm, RoPE, bf16, scattered into the paged latent cache.
//
// Bound by HBM (2,304 bytes a row of 576).  A warp walks rows `step` apart; rows and their
// cos/sin come by bulk copies into a ring of four a warp, 82 KB in flight an SM: 65,536 rows
// take 51 us with plain loads, 39 us with loads a row ahead in registers (16 warps an SM) and
// 30 us with the ring (5.4 TB/s; six or eight deep, or two CTAs an SM, the same).  Lane l holds
// dims 8l..8l+7 and 256 + 8l.. of the 512; the rotated dims are taken from the ring again, a pair
// (i, i + 32) a lane (pairs exchanged by shuffles, by eight lanes: 347 warp instructions a row and
// 36 us).
#include <algorithm>

#include "latent.cuh"
#include "mma_bf16.cuh"

namespace fp4idx {
namespace {

constexpr int kWarps = 16;
constexpr int kRing = 4;  // rows in flight a warp
constexpr int kValue = FP4IDX_LATENT_VALUE;

__device__ __forceinline__ void unpack(const uint4& u, float* v) {
  v[0] = __uint_as_float(u.x << 16); v[1] = __uint_as_float(u.x & 0xFFFF0000u);
  v[2] = __uint_as_float(u.y << 16); v[3] = __uint_as_float(u.y & 0xFFFF0000u);
  v[4] = __uint_as_float(u.z << 16); v[5] = __uint_as_float(u.z & 0xFFFF0000u);
  v[6] = __uint_as_float(u.w << 16); v[7] = __uint_as_float(u.w & 0xFFFF0000u);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint4 pack(const float* v) {
  return make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
}
__device__ __forceinline__ float bf16_at(const uint8_t* p) {
  return __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(p) << 16);
}

template <int kWidth>
struct Ring {
  static constexpr uint32_t kRow = kWidth * 2, kSlot = kRow + kRope * 2;  // the row, its cos/sin
  static constexpr uint32_t kOffBar = kWarps * kRing * kSlot;
  static constexpr uint32_t kOffAbort = kOffBar + kWarps * kRing * 8;
  static constexpr uint32_t kBytes = kOffAbort + 16;
};

template <int kWidth>
__global__ void __launch_bounds__(kWarps * 32, 1) store_latent_kernel(
    const uint16_t* kv, int64_t n_rows, const int32_t* positions,
    const int32_t* slots, const uint16_t* norm_w, float eps,
    const uint16_t* cos_sin, int32_t max_pos, uint16_t* cache, int64_t num_pages,
    int32_t* status, uint64_t wait_cycles, int32_t idle) {
  using R = Ring<kWidth>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kRot = kWidth - kRope;  // the first rotated dim
  uint8_t* ring = smem + warp * kRing * R::kSlot;
  const uint32_t bars = ptx::smem_addr(smem) + R::kOffBar + warp * kRing * 8;
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(smem + R::kOffAbort);
  if (lane == 0) {
    for (int i = 0; i < kRing; i++) ptx::mbar_init(bars + i * 8, 1);
    if (warp == 0) *abort_flag = 0;
    ptx::fence_mbar_init();
    ptx::fence_proxy_async_smem();
  }
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const pipe::Ctl ctl{abort_flag, status, wait_cycles};
  float w0[8], w1[8];
  unpack(*reinterpret_cast<const uint4*>(norm_w + lane * 8), w0);
  unpack(*reinterpret_cast<const uint4*>(norm_w + 256 + lane * 8), w1);
  // the weights of the lane's rotated pair (width 512, where those dims are normalised)
  float wp = 0.f, wq = 0.f;
  if (kWidth == 512) {
    wp = bf16_at(reinterpret_cast<const uint8_t*>(norm_w + kRot + lane));
    wq = bf16_at(reinterpret_cast<const uint8_t*>(norm_w + kRot + 32 + lane));
  }
  const int64_t step = (int64_t)gridDim.x * kWarps;
  uint32_t phases = 0;  // a bit a ring slot
  // 32 of the warp's rows at a time: lane i has the slot and position of the i-th
  for (int64_t n0 = (int64_t)blockIdx.x * kWarps + warp; n0 < n_rows; n0 += 32 * step) {
    const int64_t mine = n0 + lane * step;
    int32_t slot = -1, pos = 0;
    if (mine < n_rows) {
      slot = slots[mine];
      pos = positions[mine];
    }
    if (slot >= 0) {
      const bool bad_slot = slot >= num_pages * kPage;
      if (bad_slot || pos < 0 || pos >= max_pos) {
        record_error(status, bad_slot ? FP4IDX_ERR_BAD_PAGE : FP4IDX_ERR_BAD_POSITION);
        slot = -1;
      }
    }
    // the rows to store, in order; the i-th of them uses ring slot i % kRing
    const uint32_t todo = __ballot_sync(~0u, slot >= 0);
    const int count = __popc(todo);
    uint32_t ahead = todo;  // not asked for yet
    int asked = 0;
    const auto ask = [&]() {
      const int i = __ffs(ahead) - 1;
      ahead &= ahead - 1;
      const int32_t at = __shfl_sync(~0u, pos, i);
      if (lane == 0 && !idle) {
        const uint32_t bar = bars + (asked % kRing) * 8, dst = ptx::smem_addr(ring) + (asked % kRing) * R::kSlot;
        ptx::mbar_arrive_expect_tx(bar, R::kSlot);
        ptx::bulk_g2s(dst, kv + (n0 + i * step) * kWidth, R::kRow, bar);
        ptx::bulk_g2s(dst + R::kRow, cos_sin + (int64_t)at * kRope, kRope * 2, bar);
      }
      asked++;
    };
    for (int i = 0; i < kRing && ahead; i++) ask();
    uint32_t left = todo;
    for (int done = 0; done < count; done++) {
      const int i = __ffs(left) - 1, s = done % kRing;
      left &= left - 1;
      if (!mma::wait_warp(bars + s * 8, phases >> s & 1, ctl, false)) {
        // every copy asked for, the late one too, lands before the CTA ends
        for (int x = done; x < asked && !idle; x++) mma::wait_warp(bars + (x % kRing) * 8, phases >> (x % kRing) & 1, ctl, false);
        return;
      }
      phases ^= 1u << s;
      const uint8_t* x = ring + s * R::kSlot;
      float a[8], b[8];
      unpack(*reinterpret_cast<const uint4*>(x + lane * 16), a);
      unpack(*reinterpret_cast<const uint4*>(x + 512 + lane * 16), b);
      float p = bf16_at(x + (kRot + lane) * 2), q = bf16_at(x + (kRot + 32 + lane) * 2);
      const float c = bf16_at(x + R::kRow + lane * 2), sn = bf16_at(x + R::kRow + 64 + lane * 2);
      __syncwarp();
      if (ahead) ask();  // into the place just read
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; e++) ss += a[e] * a[e] + b[e] * b[e];
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) ss += __shfl_xor_sync(~0u, ss, d);
      const float r = __fdiv_rn(1.f, __fsqrt_rn(ss * (1.f / kValue) + eps));
#pragma unroll
      for (int e = 0; e < 8; e++) {
        a[e] = a[e] * r * w0[e];
        b[e] = b[e] * r * w1[e];
      }
      if (kWidth == 512) {
        p = p * r * wp;
        q = q * r * wq;
      }
      const uint32_t rotated = pack2(p * c - q * sn, q * c + p * sn);
      uint16_t* y = cache + (int64_t)__shfl_sync(~0u, slot, i) * kWidth;
      *reinterpret_cast<uint4*>(y + lane * 8) = pack(a);
      if (kWidth == 576 || lane < 24) *reinterpret_cast<uint4*>(y + 256 + lane * 8) = pack(b);
      y[kRot + lane] = (uint16_t)rotated;
      y[kRot + 32 + lane] = (uint16_t)(rotated >> 16);
    }
  }
}

}  // namespace

cudaError_t launch_store_latent(const uint16_t* kv, int64_t n_rows, int32_t width, const int32_t* positions,
                                const int32_t* slots, const uint16_t* norm_w, float eps, const uint16_t* cos_sin,
                                int32_t max_pos, uint16_t* cache, int64_t num_pages, int32_t* status,
                                cudaStream_t stream) {
  auto kernel = width == 576 ? store_latent_kernel<576> : store_latent_kernel<512>;
  const size_t bytes = width == 576 ? Ring<576>::kBytes : Ring<512>::kBytes;
  cudaError_t e = set_smem_attr_once(reinterpret_cast<const void*>(kernel), bytes);
  if (e != cudaSuccess) return e;
  int fit = 0;
  e = resident_ctas(reinterpret_cast<const void*>(kernel), kWarps * 32, bytes, &fit);
  if (e != cudaSuccess) return e;
  const int grid = (int)std::min<int64_t>(fit, (n_rows + kWarps - 1) / kWarps);
  return launch_early(kernel, dim3(grid), kWarps * 32, bytes, 1, stream, kv, n_rows, positions, slots, norm_w, eps, cos_sin,
                      max_pos, cache, num_pages, status, 2 * pipeline_wait_limit_ns(), pipeline_idle_producers() ? 1 : 0);
}

}  // namespace fp4idx
