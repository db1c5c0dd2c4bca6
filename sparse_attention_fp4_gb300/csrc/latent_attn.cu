// Absorbed latent attention: one latent row a token is the key of every head (all its dims)
// and their value (its first 512).
//
// A CTA per (row, head).  Its eight warps take the row's tokens in turn; a lane holds its
// share of the query and of the output, and each warp keeps a running maximum and sum
// (rescaling its output when the maximum grows), joined at the end.
#include <algorithm>

#include "launchers.cuh"

namespace fp4idx {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ void unpack(const uint4& u, float* v) {
  v[0] = __uint_as_float(u.x << 16); v[1] = __uint_as_float(u.x & 0xFFFF0000u);
  v[2] = __uint_as_float(u.y << 16); v[3] = __uint_as_float(u.y & 0xFFFF0000u);
  v[4] = __uint_as_float(u.z << 16); v[5] = __uint_as_float(u.z & 0xFFFF0000u);
  v[6] = __uint_as_float(u.w << 16); v[7] = __uint_as_float(u.w & 0xFFFF0000u);
}

template <int kWidth>
__global__ void __launch_bounds__(kWarps * 32) latent_attn_kernel(const LatentArgs a) {
  __shared__ float part_o[kWarps][512], part_m[kWarps], part_l[kWarps];
  const int t = blockIdx.x / a.heads, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int seq = a.row_seq[t];
  int n = 0, len = 0;  // entries to look at; plain context length
  if (seq < 0 || seq >= a.num_seqs) {
    if (threadIdx.x == 0) record_error(a.status, FP4IDX_ERR_BAD_PAGE);
  } else if (a.idx) {
    n = a.context_lens ? max(0, min(a.k, a.context_lens[t])) : a.k;
  } else {
    len = a.context_lens[t];
    int extra = 0;
    for (int w = 0; w < a.words; w++) {
      const uint32_t m = a.tree[(int64_t)t * a.words + w];
      if (m) extra = 32 * w + 32 - __clz(m);
    }
    if (len < 0 || (int64_t)len + extra > a.max_context) {
      if (threadIdx.x == 0) record_error(a.status, FP4IDX_ERR_BAD_LENGTH);
    } else {
      n = len + extra;
    }
  }
  float q0[8], q1[8], q2[8], o0[8] = {}, o1[8] = {};
  const uint16_t* q = a.q + (int64_t)blockIdx.x * kWidth;
  unpack(*reinterpret_cast<const uint4*>(q + lane * 8), q0);
  unpack(*reinterpret_cast<const uint4*>(q + 256 + lane * 8), q1);
  unpack(kWidth == 576 && lane < 8 ? *reinterpret_cast<const uint4*>(q + 512 + lane * 8) : make_uint4(0, 0, 0, 0), q2);
  float m = -INFINITY, l = 0.f;
  for (int i = warp; i < n; i += kWarps) {
    int pos = i;
    if (a.idx) {
      pos = a.idx[(int64_t)t * a.k + i];
      if (pos < 0) continue;
    } else if (i >= len) {
      const int j = i - len;
      if (!((a.tree[(int64_t)t * a.words + j / 32] >> (j & 31)) & 1)) continue;
    }
    if (pos / kPage >= a.max_pages) {
      if (lane == 0) record_error(a.status, FP4IDX_ERR_BAD_LENGTH);
      continue;
    }
    const int page = a.page_table[(int64_t)seq * a.max_pages + pos / kPage];
    if (page < 0 || page >= a.num_pages) {
      if (lane == 0) record_error(a.status, FP4IDX_ERR_BAD_PAGE);
      continue;
    }
    const uint16_t* k = a.cache + ((int64_t)page * kPage + pos % kPage) * kWidth;
    float k0[8], k1[8], k2[8], s = 0.f;
    unpack(*reinterpret_cast<const uint4*>(k + lane * 8), k0);
    unpack(*reinterpret_cast<const uint4*>(k + 256 + lane * 8), k1);
#pragma unroll
    for (int d = 0; d < 8; d++) s += q0[d] * k0[d] + q1[d] * k1[d];
    if (kWidth == 576 && lane < 8) {
      unpack(*reinterpret_cast<const uint4*>(k + 512 + lane * 8), k2);
#pragma unroll
      for (int d = 0; d < 8; d++) s += q2[d] * k2[d];
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
    s *= a.scale;
    const float m1 = fmaxf(m, s), keep = m1 == -INFINITY ? 1.f : expf(m - m1);
    const float p = m1 == -INFINITY ? 0.f : expf(s - m1);
    m = m1;
    l = l * keep + p;
#pragma unroll
    for (int d = 0; d < 8; d++) {
      o0[d] = o0[d] * keep + p * k0[d];
      o1[d] = o1[d] * keep + p * k1[d];
    }
  }
#pragma unroll
  for (int d = 0; d < 8; d++) {
    part_o[warp][lane * 8 + d] = o0[d];
    part_o[warp][256 + lane * 8 + d] = o1[d];
  }
  if (lane == 0) {
    part_m[warp] = m;
    part_l[warp] = l;
  }
  __syncthreads();
  float top = -INFINITY, total = 0.f;
  for (int w = 0; w < kWarps; w++) top = fmaxf(top, part_m[w]);
  for (int w = 0; w < kWarps; w++) total += part_m[w] == -INFINITY ? part_l[w] : part_l[w] * expf(part_m[w] - top);
  for (int d = threadIdx.x; d < 512; d += kWarps * 32) {
    float o = 0.f;
    for (int w = 0; w < kWarps; w++) o += part_m[w] == -INFINITY ? part_o[w][d] : part_o[w][d] * expf(part_m[w] - top);
    o = total == 0.f ? 0.f : o / total;
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(0.f), "f"(o));
    a.out[(int64_t)blockIdx.x * 512 + d] = (uint16_t)r;
  }
  if (threadIdx.x == 0 && a.lse) a.lse[blockIdx.x] = total == 0.f ? -INFINITY : top + logf(total);
}

}  // namespace

size_t latent_attn_workspace_bytes(int64_t, int32_t) { return 256; }

cudaError_t launch_latent_attn(const LatentArgs& a, int32_t width, bool, cudaStream_t stream) {
  auto kernel = width == 576 ? latent_attn_kernel<576> : latent_attn_kernel<512>;
  kernel<<<(unsigned)(a.n_rows * a.heads), kWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace fp4idx
