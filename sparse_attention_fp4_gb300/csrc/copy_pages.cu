// Copies of whole pages in several caches at once.
//
// Bound by HBM.  A page is cut into windows of up to kMost 16-byte pieces a lane, and warps take windows, all in
// flight at once: a warp's loads, then its stores, with the next window's page ids on their way.  Small
// pages (256 bytes of scales) are a short window of their own.  20,000 index pages take 29.6 us (5.9 TB/s; a CTA a page
// and cache 56), 4,001 latent pages 87 us (6.4 TB/s).
#include <algorithm>

#include "beam.cuh"

namespace fp4idx {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMost = 10;  // pieces a lane (index pages: 8, latent pages: 15 windows of 9 or 10)

struct Window {
  uint8_t* base;
  int32_t vecs, each, first;  // pieces of a page, of a window; the region's first window
};

__device__ __forceinline__ uint4 load_vec(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__global__ void __launch_bounds__(kThreads) move_pages_kernel(const int32_t* src, const int32_t* dst, int32_t n_copies,
                                                              const int32_t* count, const __grid_constant__ Regions regions,
                                                              int32_t windows, int64_t num_pages, int32_t* status) {
  __shared__ Window table[FP4IDX_COPY_MAX_REGIONS];
  const int tid = threadIdx.x, lane = tid & 31;
  for (int r = tid; r < regions.n; r += kThreads)
    table[r] = Window{regions.base[r], regions.vecs[r], regions.each[r], regions.first[r]};
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t n = count ? max(0, min(n_copies, *count)) : n_copies;
  const int64_t at = (int64_t)blockIdx.x * kWarps + (tid >> 5), step = (int64_t)gridDim.x * kWarps;
  int64_t i = at / windows;
  int32_t q = (int32_t)(at - i * windows);
  const int64_t step_i = step / windows;
  const int32_t step_q = (int32_t)(step - step_i * windows);
  int32_t s = -1, d = -1;
  if (i < n) s = src[i], d = dst[i];
  while (i < n) {
    // the next window's ids
    int64_t next = i + step_i;
    int32_t next_q = q + step_q;
    if (next_q >= windows) next_q -= windows, next++;
    int32_t next_s = -1, next_d = -1;
    if (next < n) next_s = src[next], next_d = dst[next];
    if (s >= num_pages || d >= num_pages) {
      if (lane == 0 && s >= 0 && d >= 0) record_error(status, FP4IDX_ERR_BAD_PAGE);
    } else if (s >= 0 && d >= 0) {
      int r = -1;  // the last region whose first window is not behind q
      for (int b = 0; b < regions.n; b += 32) r += __popc(__ballot_sync(~0u, b + lane < regions.n && table[min(b + lane, regions.n - 1)].first <= q));
      const Window w = table[r];
      const int32_t v0 = (q - w.first) * w.each + lane, end = min(w.vecs, (q - w.first + 1) * w.each);
      const uint4* from = reinterpret_cast<const uint4*>(w.base) + (int64_t)s * w.vecs;
      uint4* to = reinterpret_cast<uint4*>(w.base) + (int64_t)d * w.vecs;
      uint4 v[kMost];
#pragma unroll
      for (int j = 0; j < kMost; j++)
        if (v0 + j * 32 < end) v[j] = load_vec(from + v0 + j * 32);
#pragma unroll
      for (int j = 0; j < kMost; j++)
        if (v0 + j * 32 < end) to[v0 + j * 32] = v[j];
    }
    i = next, q = next_q, s = next_s, d = next_d;
  }
}

}  // namespace

cudaError_t launch_move_pages(const int32_t* src, const int32_t* dst, int64_t n_copies, const int32_t* count,
                              Regions& regions, int64_t num_pages, int32_t* status, cudaStream_t stream) {
  int64_t windows = 0;
  for (int32_t r = 0; r < regions.n; r++) {
    const int32_t of = (regions.vecs[r] + 32 * kMost - 1) / (32 * kMost);
    regions.each[r] = (regions.vecs[r] + of - 1) / of;
    regions.first[r] = (int32_t)windows;
    windows += of;
  }
  int ctas = 0;
  const cudaError_t e = resident_ctas(reinterpret_cast<const void*>(move_pages_kernel), kThreads, 0, &ctas);
  if (e != cudaSuccess) return e;
  // four times the CTAs that run at once: the later ones begin as others end (latent pages 92 us with as many as run at
  // once, 87 with four times as many, 85 with a CTA for every eight windows; index pages 30.5, 29.6 and 31.5), and few are
  // launched for nothing where *count is far below n_copies
  const int64_t need = (n_copies * windows + kWarps - 1) / kWarps;
  return launch_early(move_pages_kernel, dim3((unsigned)std::min<int64_t>(need, 4 * (int64_t)ctas)), kThreads, 0, 1, stream, src, dst,
                      (int32_t)n_copies, count, regions, (int32_t)windows, num_pages, status);
}

}  // namespace fp4idx
