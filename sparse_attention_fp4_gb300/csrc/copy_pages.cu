// Copies of whole pages in several caches at once.
#include <algorithm>

#include "beam.cuh"

namespace fp4idx {
namespace {

constexpr int kThreads = 256;

// One CTA a (pair, region), all of them dealt out over the grid.
__global__ void __launch_bounds__(kThreads) move_pages_kernel(const int32_t* src, const int32_t* dst, int32_t n_copies,
                                                              const int32_t* count, const __grid_constant__ Regions regions,
                                                              int64_t num_pages, int32_t* status) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int32_t n = count ? max(0, min(n_copies, *count)) : n_copies;
  for (int64_t u = blockIdx.x; u < (int64_t)n * regions.n; u += gridDim.x) {
    const int i = (int)(u / regions.n), r = (int)(u - (int64_t)i * regions.n);
    const int32_t s = src[i], d = dst[i];
    if (s < 0 || d < 0) continue;
    if (s >= num_pages || d >= num_pages) {
      if (threadIdx.x == 0) record_error(status, FP4IDX_ERR_BAD_PAGE);
      continue;
    }
    const int32_t vecs = regions.vecs[r];
    const uint4* from = reinterpret_cast<const uint4*>(regions.base[r]) + (int64_t)s * vecs;
    uint4* to = reinterpret_cast<uint4*>(regions.base[r]) + (int64_t)d * vecs;
    for (int v = threadIdx.x; v < vecs; v += kThreads) to[v] = from[v];
  }
}

}  // namespace

cudaError_t launch_move_pages(const int32_t* src, const int32_t* dst, int64_t n_copies, const int32_t* count,
                              const Regions& regions, int64_t num_pages, int32_t* status, cudaStream_t stream) {
  const int64_t units = n_copies * regions.n;
  return launch_early(move_pages_kernel, dim3((unsigned)std::min<int64_t>(units, 1 << 16)), kThreads, 0, 1, stream, src, dst,
                      (int32_t)n_copies, count, regions, num_pages, status);
}

}  // namespace fp4idx
