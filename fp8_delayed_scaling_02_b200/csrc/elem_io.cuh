// Element loads of bf16 / fp16 / fp32 tensors at any element alignment, and
// byte stores at any alignment, shared by the streaming kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace fp8ds {

template <int DT> struct In;
template <> struct In<FP8_IN_BF16> { static constexpr int kBytes = 2; };
template <> struct In<FP8_IN_FP16> { static constexpr int kBytes = 2; };
template <> struct In<FP8_IN_FP32> { static constexpr int kBytes = 4; };

template <int DT>
__device__ __forceinline__ float load_one(const uint8_t* p) {
  if constexpr (DT == FP8_IN_BF16) {
    return __uint_as_float(uint32_t(*reinterpret_cast<const uint16_t*>(p)) << 16);
  } else if constexpr (DT == FP8_IN_FP16) {
    return __half2float(__ushort_as_half(*reinterpret_cast<const uint16_t*>(p)));
  } else {
    return *reinterpret_cast<const float*>(p);
  }
}

// Two 16-bit elements packed in one word -> floats (low half first).
template <int DT>
__device__ __forceinline__ void unpack2(uint32_t w, float& lo, float& hi) {
  if constexpr (DT == FP8_IN_BF16) {
    lo = __uint_as_float(w << 16);
    hi = __uint_as_float(w & 0xFFFF0000u);
  } else {
    __half2 h = *reinterpret_cast<__half2*>(&w);
    float2 f = __half22float2(h);
    lo = f.x;
    hi = f.y;
  }
}

__device__ __forceinline__ uint4 ldg16(const uint8_t* p) {
  return __ldg(reinterpret_cast<const uint4*>(p));
}

// Words [0, NW) of the byte stream that starts `ph` bytes past the 16-byte
// aligned address `q`, given the aligned words W[0, NW + 4).  ph is a multiple
// of the element size; the word shift is selected without dynamic register
// indexing and the half-word remainder (16-bit types only) is a funnel shift.
template <int NW>
__device__ __forceinline__ void realign(const uint32_t (&W)[NW + 4], int ph, uint32_t (&D)[NW]) {
  const int ws = ph >> 2;
  uint32_t X[NW + 1];
#pragma unroll
  for (int i = 0; i <= NW; ++i) {
    uint32_t a = W[i], b = W[i + 1], c = W[i + 2], d = W[i + 3];
    X[i] = ws == 0 ? a : (ws == 1 ? b : (ws == 2 ? c : d));
  }
  const bool half = (ph & 2) != 0;
#pragma unroll
  for (int i = 0; i < NW; ++i) D[i] = half ? __funnelshift_r(X[i], X[i + 1], 16) : X[i];
}

// Load N (8 or 16) consecutive elements starting at element address p into v.
// Only 16-byte granules that hold at least one of the N elements are read.
template <int DT, int N>
__device__ __forceinline__ void load_vec(const uint8_t* p, float (&v)[N]) {
  constexpr int kB = In<DT>::kBytes;
  constexpr int NW = N * kB / 4;      // useful words
  constexpr int NG = NW / 4;          // useful granules when aligned
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  const int ph = int(a & 15);
  const uint8_t* q = p - ph;
  uint32_t W[NW + 4];
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    uint4 t = ldg16(q + 16 * g);
    W[4 * g] = t.x; W[4 * g + 1] = t.y; W[4 * g + 2] = t.z; W[4 * g + 3] = t.w;
  }
  if (ph != 0) {
    uint4 t = ldg16(q + 16 * NG);
    W[4 * NG] = t.x; W[4 * NG + 1] = t.y; W[4 * NG + 2] = t.z; W[4 * NG + 3] = t.w;
  } else {
    W[4 * NG] = W[4 * NG + 1] = W[4 * NG + 2] = W[4 * NG + 3] = 0u;
  }
  uint32_t D[NW];
  realign<NW>(W, ph, D);
  if constexpr (kB == 2) {
#pragma unroll
    for (int i = 0; i < NW; ++i) unpack2<DT>(D[i], v[2 * i], v[2 * i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < NW; ++i) v[i] = __uint_as_float(D[i]);
  }
}

// Aligned fast path (p is 16-byte aligned).
template <int DT, int N>
__device__ __forceinline__ void load_vec_aligned(const uint8_t* p, float (&v)[N]) {
  constexpr int kB = In<DT>::kBytes;
  constexpr int NW = N * kB / 4;
#pragma unroll
  for (int g = 0; g < NW / 4; ++g) {
    uint4 t = ldg16(p + 16 * g);
    uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (kB == 2) {
        unpack2<DT>(w[i], v[8 * g + 2 * i], v[8 * g + 2 * i + 1]);
      } else {
        v[4 * g + i] = __uint_as_float(w[i]);
      }
    }
  }
}

// Eight bytes (lo, hi) to an address of any alignment with the widest
// aligned stores it allows.
__device__ __forceinline__ void store8_any(uint8_t* o, uint32_t lo, uint32_t hi) {
  const int m = int(reinterpret_cast<uintptr_t>(o) & 7);
  if (m == 0) {
    *reinterpret_cast<uint2*>(o) = make_uint2(lo, hi);
  } else if (m == 4) {
    reinterpret_cast<uint32_t*>(o)[0] = lo;
    reinterpret_cast<uint32_t*>(o)[1] = hi;
  } else if ((m & 1) == 0) {
    uint16_t* h = reinterpret_cast<uint16_t*>(o);
    h[0] = uint16_t(lo);
    h[1] = uint16_t(lo >> 16);
    h[2] = uint16_t(hi);
    h[3] = uint16_t(hi >> 16);
  } else {
    o[0] = uint8_t(lo);
    uint16_t* h = reinterpret_cast<uint16_t*>(o + 1);
    h[0] = uint16_t(__byte_perm(lo, 0, 0x0021));
    h[1] = uint16_t(__byte_perm(lo, hi, 0x0043));
    h[2] = uint16_t(__byte_perm(hi, 0, 0x0021));
    o[7] = uint8_t(hi >> 24);
  }
}

}  // namespace fp8ds
