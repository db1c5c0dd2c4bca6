// Expanded latent attention: causal attention over packed prompts, per-head keys (128 own
// dims and 64 rotated ones that the heads share) and values (128 dims).
//
// A warp per (query row, head); a lane holds six dims of the query and four of the output.
#include <algorithm>

#include "launchers.cuh"

namespace fp4idx {
namespace {

constexpr int kWarps = 8;
constexpr int kKey = FP4IDX_PREFILL_KEY, kVal = FP4IDX_PREFILL_VALUE;

__device__ __forceinline__ float2 two(const uint16_t* p) {
  const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
}

__global__ void __launch_bounds__(kWarps * 32) latent_prefill_kernel(const PrefillArgs a) {
  const int seq = blockIdx.z, h = blockIdx.y, lane = threadIdx.x & 31;
  const int64_t q0 = a.cu_q[seq], q1 = a.cu_q[seq + 1], k0 = a.cu_kv[seq], k1 = a.cu_kv[seq + 1];
  if (q0 < 0 || q1 < q0 || q1 > a.n_q || k0 < 0 || k1 < k0 || k1 > a.n_kv || q1 - q0 > a.max_q || k1 - k0 > a.max_kv) {
    if (threadIdx.x == 0) record_error(a.status, FP4IDX_ERR_BAD_LENGTH);
    return;
  }
  const int i = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (i >= q1 - q0) return;
  const int64_t row = (q0 + i) * a.heads + h;
  const uint16_t* q = a.q + row * kKey;
  const float2 qa = two(q + lane * 4), qb = two(q + lane * 4 + 2), qc = two(q + 128 + lane * 2);
  const int64_t n = (k1 - k0) - (q1 - q0) + i + 1;
  float m = -INFINITY, l = 0.f, o[4] = {};
  for (int64_t j = k0; j < k0 + n; j++) {
    const uint16_t* kv = a.kv + (j * a.heads + h) * 256;
    const float2 ka = two(kv + lane * 4), kb = two(kv + lane * 4 + 2), kc = two(a.k_rope + j * 64 + lane * 2);
    const float2 va = two(kv + 128 + lane * 4), vb = two(kv + 128 + lane * 4 + 2);
    float s = qa.x * ka.x + qa.y * ka.y + qb.x * kb.x + qb.y * kb.y + qc.x * kc.x + qc.y * kc.y;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
    s *= a.scale;
    const float m1 = fmaxf(m, s), keep = m1 == -INFINITY ? 1.f : expf(m - m1);
    const float p = m1 == -INFINITY ? 0.f : expf(s - m1);
    m = m1;
    l = l * keep + p;
    o[0] = o[0] * keep + p * va.x;
    o[1] = o[1] * keep + p * va.y;
    o[2] = o[2] * keep + p * vb.x;
    o[3] = o[3] * keep + p * vb.y;
  }
  const float r = l == 0.f ? 0.f : 1.f / l;
  uint2 u;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u.x) : "f"(o[1] * r), "f"(o[0] * r));
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u.y) : "f"(o[3] * r), "f"(o[2] * r));
  *reinterpret_cast<uint2*>(a.out + row * kVal + lane * 4) = u;
  if (lane == 0 && a.lse) a.lse[row] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace

cudaError_t launch_latent_prefill(const PrefillArgs& a, cudaStream_t stream) {
  const dim3 grid((a.max_q + kWarps - 1) / kWarps, a.heads, a.n_seqs);
  latent_prefill_kernel<<<grid, kWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace fp4idx
