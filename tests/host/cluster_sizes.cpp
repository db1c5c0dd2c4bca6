// How many clusters fit, over a CUDA runtime that answers as this file says: a size that the
// device cannot place counts as none that fit, any other failure is the call's.
#include <cuda_runtime_api.h>

#include <cstdio>

namespace fp4idx {
cudaError_t resident_clusters(const void* kernel, int size, int threads, size_t smem, int* out);
}

namespace {
int occupancy_calls = 0, attribute_calls = 0, left_over = 0;
cudaError_t occupancy_answer = cudaSuccess, attribute_answer = cudaSuccess;
int clusters = 0;
cudaError_t answer(cudaError_t e) {
  if (e != cudaSuccess) left_over = e;
  return e;
}
}  // namespace

extern "C" {
cudaError_t cudaGetDevice(int* d) { *d = 0; return cudaSuccess; }
cudaError_t cudaGetLastError() { const int e = left_over; left_over = 0; return (cudaError_t)e; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) { *v = 152; return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { attribute_calls++; return answer(attribute_answer); }
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessor(int* n, const void*, int, size_t) { *n = 1; return cudaSuccess; }
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t*) {
  occupancy_calls++;
  *n = clusters;
  return answer(occupancy_answer);
}
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void**, unsigned int, unsigned long long, cudaDriverEntryPointQueryResult*) {
  return cudaErrorNotSupported;
}
void** __cudaRegisterFatBinary(void*) { return nullptr; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
}

#define CHECK(x)                                       \
  do {                                                 \
    if (!(x)) {                                        \
      std::printf("line %d: %s\n", __LINE__, #x);      \
      return 1;                                        \
    }                                                  \
  } while (0)

int main() {
  static const char kernels[8] = {};
  int fit = -1;
  // a size that fits, asked once
  clusters = 9;
  CHECK(fp4idx::resident_clusters(kernels + 0, 8, 640, 200000, &fit) == cudaSuccess && fit == 9);
  CHECK(fp4idx::resident_clusters(kernels + 0, 8, 640, 200000, &fit) == cudaSuccess && fit == 9 && occupancy_calls == 1);
  // sizes that the device cannot place: none fit, asked once, no error left behind
  const cudaError_t cannot[] = {cudaErrorInvalidClusterSize, cudaErrorInvalidConfiguration, cudaErrorInvalidValue, cudaErrorNotSupported};
  for (int i = 0; i < 4; i++) {
    occupancy_answer = cannot[i];
    fit = -1;
    occupancy_calls = 0;
    for (int again = 0; again < 2; again++)
      CHECK(fp4idx::resident_clusters(kernels + 1 + i, 8, 640, 200000, &fit) == cudaSuccess && fit == 0);
    CHECK(occupancy_calls == 1 && left_over == 0);
  }
  // a device that refuses sizes above the portable one: none fit, and the smaller one still does
  occupancy_answer = cudaSuccess;
  attribute_answer = cudaErrorInvalidValue;
  CHECK(fp4idx::resident_clusters(kernels + 5, 16, 640, 200000, &fit) == cudaSuccess && fit == 0 && left_over == 0);
  attribute_calls = 0;
  CHECK(fp4idx::resident_clusters(kernels + 5, 8, 640, 200000, &fit) == cudaSuccess && fit == 9 && attribute_calls == 0);
  // any other failure is reported, and asked again the next time
  attribute_answer = cudaSuccess;
  occupancy_answer = cudaErrorMemoryAllocation;
  CHECK(fp4idx::resident_clusters(kernels + 6, 4, 640, 200000, &fit) == cudaErrorMemoryAllocation);
  occupancy_answer = cudaSuccess;
  CHECK(fp4idx::resident_clusters(kernels + 6, 4, 640, 200000, &fit) == cudaSuccess && fit == 9);
  std::printf("OK\n");
  return 0;
}
