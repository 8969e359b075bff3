// Host-side launch helpers of the streaming kernels.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

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

// Whether p lies on a multiple of `a` bytes (a null pointer does).
inline bool on(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// An argument's memory.  `over`: an output that may be exactly the memory of
// an input marked `under` (each element is read before its place is written,
// by the same thread); every other overlap with an output is a mistake.
struct Span {
  const void* p;
  size_t n;
  bool out, over, under;
};

inline bool spans_clash(const Span* s, int n) {
  for (int i = 0; i < n; ++i) {
    if (!s[i].out || s[i].p == nullptr || s[i].n == 0) continue;
    for (int j = 0; j < n; ++j) {
      if (j == i || s[j].p == nullptr || s[j].n == 0) continue;
      const uintptr_t a = reinterpret_cast<uintptr_t>(s[i].p), b = reinterpret_cast<uintptr_t>(s[j].p);
      if (a >= b + s[j].n || b >= a + s[i].n) continue;
      if (s[i].over && s[j].under && a == b && s[i].n == s[j].n) continue;
      return true;
    }
  }
  return false;
}

}  // namespace fp8ds
