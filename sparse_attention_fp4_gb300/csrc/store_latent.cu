// Latent store: RMSNorm, RoPE, bf16, scattered into the paged latent cache.
//
// A warp per row.  Lane l holds dims 8l..8l+7 and 256 + 8l.. of the 512, and at width 576
// lanes 0..7 hold the last 64; the two halves of a RoPE pair (i, i + 32) are then four lanes
// apart.
#include <algorithm>

#include "launchers.cuh"

namespace fp4idx {
namespace {

constexpr int kWarps = 8;
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
// The eight lanes of a rotated run of 64 dims: lane r of the run holds dims 8r..8r+7, its
// pair's other half four lanes away.  Every lane of the warp takes part in the shuffles.
__device__ __forceinline__ void rope(float* v, int r, const uint4& uc, const uint4& us, bool rotate) {
  float c[8], s[8];
  unpack(uc, c);
  unpack(us, s);
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const float other = __shfl_xor_sync(~0u, v[i], 4);
    if (rotate) v[i] = r < 4 ? v[i] * c[i] - other * s[i] : v[i] * c[i] + other * s[i];
  }
}

// A warp walks rows `step` apart.  The row's values and its cos/sin are loaded a row ahead,
// its slot and position two rows ahead, so that no load waits for another.
template <int kWidth>
__global__ void __launch_bounds__(kWarps * 32) store_latent_kernel(
    const uint16_t* __restrict__ kv, int64_t n_rows, const int32_t* __restrict__ positions,
    const int32_t* __restrict__ slots, const uint16_t* __restrict__ norm_w, float eps,
    const uint16_t* __restrict__ cos_sin, int32_t max_pos, uint16_t* __restrict__ cache, int64_t num_pages,
    int32_t* status) {
  const int lane = threadIdx.x & 31;
  const bool rotates = kWidth == 576 ? lane < 8 : lane >= 24;
  float w0[8], w1[8];
  unpack(*reinterpret_cast<const uint4*>(norm_w + lane * 8), w0);
  unpack(*reinterpret_cast<const uint4*>(norm_w + 256 + lane * 8), w1);
  struct Meta {
    int32_t slot, pos;
  };
  struct Data {
    uint4 a, b, t, c, s;
  };
  const uint4 none = make_uint4(0, 0, 0, 0);
  const auto meta = [&](int64_t n) {
    return n < n_rows ? Meta{__ldg(slots + n), __ldg(positions + n)} : Meta{-1, 0};
  };
  const auto data = [&](int64_t n, const Meta& m) {
    Data d{none, none, none, none, none};
    if (m.slot < 0) return d;
    const uint16_t* x = kv + n * kWidth;
    d.a = __ldcs(reinterpret_cast<const uint4*>(x + lane * 8));
    d.b = __ldcs(reinterpret_cast<const uint4*>(x + 256 + lane * 8));
    if (kWidth == 576 && rotates) d.t = __ldcs(reinterpret_cast<const uint4*>(x + 512 + lane * 8));
    if (rotates && m.pos >= 0 && m.pos < max_pos) {
      const uint16_t* cs = cos_sin + (int64_t)m.pos * kRope + (lane & 3) * 8;
      d.c = __ldg(reinterpret_cast<const uint4*>(cs));
      d.s = __ldg(reinterpret_cast<const uint4*>(cs + 32));
    }
    return d;
  };
  const int64_t step = (int64_t)gridDim.x * kWarps;
  int64_t n = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  Meta m = meta(n), m1 = meta(n + step);
  Data d = data(n, m);
  for (; n < n_rows; n += step) {
    const Data d1 = data(n + step, m1);
    const Meta m2 = meta(n + 2 * step);
    const bool bad_slot = m.slot >= num_pages * kPage, bad_pos = m.pos < 0 || m.pos >= max_pos;
    if (m.slot >= 0 && (bad_slot || bad_pos)) {
      if (lane == 0) record_error(status, bad_slot ? FP4IDX_ERR_BAD_PAGE : FP4IDX_ERR_BAD_POSITION);
    } else if (m.slot >= 0) {
      float a[8], b[8], t[8];
      unpack(d.a, a);
      unpack(d.b, b);
      if (kWidth == 576) unpack(d.t, t);
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; i++) ss += a[i] * a[i] + b[i] * b[i];
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) ss += __shfl_xor_sync(~0u, ss, x);
      const float r = __fdiv_rn(1.f, __fsqrt_rn(ss * (1.f / kValue) + eps));
#pragma unroll
      for (int i = 0; i < 8; i++) {
        a[i] = a[i] * r * w0[i];
        b[i] = b[i] * r * w1[i];
      }
      uint16_t* y = cache + (int64_t)m.slot * kWidth;
      rope(kWidth == 576 ? t : b, lane & 7, d.c, d.s, rotates);
      if (kWidth == 576 && rotates) *reinterpret_cast<uint4*>(y + 512 + lane * 8) = pack(t);
      *reinterpret_cast<uint4*>(y + lane * 8) = pack(a);
      *reinterpret_cast<uint4*>(y + 256 + lane * 8) = pack(b);
    }
    d = d1;
    m = m1;
    m1 = m2;
  }
}

}  // namespace

cudaError_t launch_store_latent(const uint16_t* kv, int64_t n_rows, int32_t width, const int32_t* positions,
                                const int32_t* slots, const uint16_t* norm_w, float eps, const uint16_t* cos_sin,
                                int32_t max_pos, uint16_t* cache, int64_t num_pages, int32_t* status,
                                cudaStream_t stream) {
  auto kernel = width == 576 ? store_latent_kernel<576> : store_latent_kernel<512>;
  int fit = 0;
  cudaError_t e = resident_ctas(reinterpret_cast<const void*>(kernel), kWarps * 32, 0, &fit);
  if (e != cudaSuccess) return e;
  const int grid = (int)std::min<int64_t>(fit, (n_rows + kWarps - 1) / kWarps);
  kernel<<<grid, kWarps * 32, 0, stream>>>(kv, n_rows, positions, slots, norm_w, eps, cos_sin, max_pos, cache,
                                           num_pages, status);
  return cudaGetLastError();
}

}  // namespace fp4idx
