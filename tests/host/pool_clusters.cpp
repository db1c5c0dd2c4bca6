// The clusters of a fork and of a compaction, over a CUDA runtime that answers as this file says: sixteen CTAs where
// the device places them, else eight where the pool's marks have room in eight.
#include <cuda_runtime_api.h>

#include <cstdio>
#include <cstring>
#include <initializer_list>

#include "fp4idx.h"

namespace {
int places_sixteen = 1, launches = 0, left_over = 0;
struct Launch {
  unsigned ctas = 0, cluster = 0;
  size_t smem = 0;
  int shift = 0;
  bool full = false;
} last;
cudaError_t answer(cudaError_t e) {
  if (e != cudaSuccess) left_over = e;
  return e;
}
}  // namespace

extern "C" {
cudaError_t cudaGetDevice(int* d) { *d = places_sixteen; return cudaSuccess; }  // (what is known of one device is not asked again)
cudaError_t cudaGetLastError() { const int e = left_over; left_over = 0; return (cudaError_t)e; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) { *v = 152; return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessor(int* n, const void*, int, size_t) { *n = 1; return cudaSuccess; }
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t* c) {
  const bool large = c->attrs[0].val.clusterDim.x > 8;
  *n = large && !places_sixteen ? 0 : 4;
  return answer(large && !places_sixteen ? cudaErrorInvalidClusterSize : cudaSuccess);
}
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void**, unsigned int, unsigned long long, cudaDriverEntryPointQueryResult*) {
  return cudaErrorNotSupported;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void*, void** args) {
  last = Launch{};
  last.ctas = c->gridDim.x;
  last.smem = c->dynamicSmemBytes;
  last.cluster = 1;
  for (unsigned i = 0; i < c->numAttrs; i++)
    if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) last.cluster = c->attrs[i].val.clusterDim.x;
  std::memcpy(&last.shift, args[1], sizeof(int));
  std::memcpy(&last.full, args[2], sizeof(bool));
  launches++;
  return last.cluster > 8 && !places_sixteen ? answer(cudaErrorInvalidClusterSize) : cudaSuccess;
}
// (launches in the other form, of which there is none)
cudaError_t __cudaLaunchKernel(cudaKernel_t, dim3, dim3, void**, size_t, cudaStream_t) { return cudaErrorNotSupported; }
cudaError_t __cudaGetKernel(cudaKernel_t*, const void*) { return cudaErrorNotSupported; }
cudaError_t __cudaPopCallConfiguration(dim3*, dim3*, size_t*, void*) { return cudaErrorNotSupported; }
void** __cudaRegisterFatBinary(void*) { return nullptr; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char*, char*, const char*, int, uint3*, uint3*, dim3*, dim3*, int*) {}
}

#define CHECK(x)                                                                                          \
  do {                                                                                                    \
    if (!(x)) {                                                                                           \
      std::printf("line %d: %s (pool %lld, %d rows, %d x %u CTAs)\n", __LINE__, #x, (long long)pool, rows, launches, last.ctas); \
      return 1;                                                                                           \
    }                                                                                                     \
  } while (0)

int main() {
  int32_t *at = reinterpret_cast<int32_t*>(1 << 20), *out = reinterpret_cast<int32_t*>(1 << 21);  // (nothing reads them)
  const int64_t pools[] = {1, 33, 5000, 241000, 1 << 19, (1 << 19) + 1, 1 << 20, 1 << 21, 1 << 22, (1 << 22) + 1, 1 << 23};
  for (int64_t pool : pools)
    for (int rows : {1, 40, 8192})
      for (int fork = 0; fork < 2; fork++) {
        int rc[2];
        Launch of[2];
        for (int s = 0; s < 2; s++) {
          places_sixteen = s;
          launches = 0;
          rc[s] = fork ? fp4idx_fork_pages(at, at, rows, 900, 1, at, rows, pool, nullptr, at, 9, nullptr, out, out, at, at, at, nullptr, nullptr)
                       : fp4idx_compact_pages(at, at, rows, 900, 1, pool, nullptr, at, (size_t)1 << 30, at, 9, out, at, at, 4, at, nullptr, nullptr);
          of[s] = last;
          CHECK(left_over == 0);
          CHECK(launches == (rc[s] == FP4IDX_OK));
        }
        // sixteen wherever they are placed and the call has work or a pool for them, as ever
        CHECK(rc[1] == FP4IDX_OK);
        const bool large = (int64_t)rows * 900 * (fork ? 2 : 1) > 8 * 2048 || pool > (1 << 19);
        CHECK((of[1].cluster == 16) == large);
        // else eight: every pool whose marks eight CTAs hold; the marks lie within the memory that the launch has
        if (rc[0] != FP4IDX_OK) {
          CHECK(rc[0] == FP4IDX_ERR_CUDA && pool > (1 << 22));
          continue;
        }
        for (int s = 0; s < 2; s++) {
          const Launch& l = of[s];
          last = l;
          CHECK(l.ctas == l.cluster && l.cluster <= (s ? 16 : 8));
          const int64_t words = (pool + 31) / 32, share = (int64_t)1 << l.shift;
          CHECK(share * l.ctas >= words);
          const int64_t marks = 4 * (fork ? 2 : 1) * share * (l.full ? l.ctas : 1) + (fork ? 12 * rows : 4 * share);
          CHECK((int64_t)l.smem == marks && marks <= 225 * 1024);
        }
        if (!large) CHECK(of[0].cluster == of[1].cluster && of[0].smem == of[1].smem);
      }
  std::printf("OK\n");
  return 0;
}
