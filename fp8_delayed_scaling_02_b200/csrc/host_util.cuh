// Host-side launch helpers of the streaming kernels.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "fp8ds.h"

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

inline bool overlap(const void* p, size_t n, const void* q, size_t m) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return p != nullptr && q != nullptr && n != 0 && m != 0 && a < b + m && b < a + n;
}

// The words of a ring, and of an amax beside it, that a call reads and writes.
struct RingWords {
  const void* p[6];
  RingWords(const fp8_ring& r, const float* amax_out)
      : p{r.history, r.idx, r.scale, r.scale_inv, r.scratch, amax_out} {}
  static size_t bytes(int i) { return i == 0 ? 64 : i == 4 ? 16 : 4; }
  bool aligned() const { return on(p[0], 4) && on(p[1], 4) && on(p[2], 4) && on(p[3], 4) && on(p[5], 4); }
  // Whether a word lies in one of the other arguments, or the amax in the ring.
  bool clash(const Span* s, int n) const {
    for (int i = 0; i < 6; ++i) {
      for (int j = 0; j < n; ++j)
        if (overlap(p[i], bytes(i), s[j].p, s[j].n)) return true;
      if (i < 5 && overlap(p[i], bytes(i), p[5], 4)) return true;
    }
    return false;
  }
  bool clash(const RingWords& o) const {
    for (int i = 0; i < 6; ++i)
      for (int j = 0; j < 6; ++j)
        if (overlap(p[i], bytes(i), o.p[j], bytes(j))) return true;
    return false;
  }
};

inline bool spans_clash(const Span* s, int n) {
  for (int i = 0; i < n; ++i) {
    if (!s[i].out || s[i].p == nullptr || s[i].n == 0) continue;
    for (int j = 0; j < n; ++j) {
      if (j == i || !overlap(s[i].p, s[i].n, s[j].p, s[j].n)) continue;
      if (s[i].over && s[j].under && s[i].p == s[j].p && s[i].n == s[j].n) continue;
      return true;
    }
  }
  return false;
}

}  // namespace fp8ds
