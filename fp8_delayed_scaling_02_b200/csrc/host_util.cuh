// Host-side launch helpers of the streaming kernels.
#pragma once

#include <cuda_runtime.h>

namespace fp8ds {

inline int sm_count_current() {
  static int cached[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return -1;
  if (dev < 0 || dev >= 64) return -1;
  if (cached[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return -1;
    cached[dev] = n;
  }
  return cached[dev];
}

// Resident blocks per SM of a kernel without dynamic shared memory (cached
// per device by the caller's static array).
template <typename Kern>
int resident_blocks(Kern kern, int threads, int (&cached)[64]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return -1;
  if (cached[dev] == 0) {
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, threads, 0) != cudaSuccess || n < 1) return -1;
    cached[dev] = n;
  }
  return cached[dev];
}

}  // namespace fp8ds
