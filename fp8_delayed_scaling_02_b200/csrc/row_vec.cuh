// Eight consecutive elements of a row, kept packed in registers as they lie in
// memory, for kernels whose threads own fixed columns of a row-major tensor.
//
// kAligned: the tensor's base is 16-byte aligned and its width a multiple of
// 8, so every vector is one 16-byte access (two for float32).  Otherwise rows
// start at any element alignment: loads read the aligned 16-byte granules that
// hold the elements and shift, stores use the widest pieces the address allows,
// and a row's last, partial vector goes element by element.
// Plain loads (not the read-only path): callers may write in place.
#pragma once

#include "common.cuh"
#include "elem_io.cuh"

namespace fp8ds {

template <int DT>
struct Vec8 {
  static constexpr int kWords = In<DT>::kBytes * 2;
  uint32_t w[kWords];
};

__device__ __forceinline__ uint4 ld16(const uint8_t* p) { return *reinterpret_cast<const uint4*>(p); }

// The NW words that start ph (a multiple of 2, below 16) bytes into W.
template <int NW>
__device__ __forceinline__ void shift_down(uint32_t (&W)[NW + 4], int ph, uint32_t* out) {
#pragma unroll
  for (int i = 0; i < NW + 2; ++i) W[i] = ph & 8 ? W[i + 2] : W[i];
#pragma unroll
  for (int i = 0; i < NW + 1; ++i) W[i] = ph & 4 ? W[i + 1] : W[i];
  const int s = 8 * (ph & 2);
#pragma unroll
  for (int i = 0; i < NW; ++i) out[i] = __funnelshift_r(W[i], W[i + 1], s);
}

// Elements c .. c+7 of a row of `cols`; zeros beyond its end.
template <int DT, bool kAligned>
__device__ __forceinline__ Vec8<DT> load8(const uint8_t* row, int c, int cols) {
  constexpr int kB = In<DT>::kBytes;
  constexpr int NW = Vec8<DT>::kWords, NG = NW / 4;
  Vec8<DT> r;
#pragma unroll
  for (int i = 0; i < NW; ++i) r.w[i] = 0u;
  if (c >= cols) return r;
  const uint8_t* p = row + int64_t(c) * kB;
  const int ph = int(reinterpret_cast<uintptr_t>(p) & 15);
  if (kAligned || (c + 8 <= cols && ph == 0)) {
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const uint4 t = ld16(p + 16 * g);
      r.w[4 * g] = t.x; r.w[4 * g + 1] = t.y; r.w[4 * g + 2] = t.z; r.w[4 * g + 3] = t.w;
    }
    return r;
  }
  if constexpr (!kAligned) {
    if (c + 8 <= cols) {
      const uint8_t* q = p - ph;
      uint32_t W[NW + 4];
#pragma unroll
      for (int g = 0; g <= NG; ++g) {
        const uint4 t = ld16(q + 16 * g);
        W[4 * g] = t.x; W[4 * g + 1] = t.y; W[4 * g + 2] = t.z; W[4 * g + 3] = t.w;
      }
      shift_down<NW>(W, ph, r.w);
      return r;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (c + i < cols) {
        if constexpr (kB == 2) r.w[i >> 1] |= uint32_t(reinterpret_cast<const uint16_t*>(p)[i]) << (16 * (i & 1));
        else r.w[i] = reinterpret_cast<const uint32_t*>(p)[i];
      }
    }
  }
  return r;
}

template <int DT>
__device__ __forceinline__ void unpack8(const Vec8<DT>& r, float (&v)[8]) {
  if constexpr (In<DT>::kBytes == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack2<DT>(r.w[i], v[2 * i], v[2 * i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r.w[i]);
  }
}

// Each value rounded once, to nearest even, to the element type.
template <int DT>
__device__ __forceinline__ Vec8<DT> pack8(const float (&v)[8]) {
  Vec8<DT> r;
  if constexpr (DT == FP8_IN_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      r.w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  } else if constexpr (DT == FP8_IN_FP16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      r.w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.w[i] = __float_as_uint(v[i]);
  }
  return r;
}

template <int DT, bool kAligned>
__device__ __forceinline__ void store8(uint8_t* row, int c, int cols, const Vec8<DT>& r) {
  constexpr int kB = In<DT>::kBytes;
  constexpr int NW = Vec8<DT>::kWords, NG = NW / 4;
  if (c >= cols) return;
  uint8_t* p = row + int64_t(c) * kB;
  const uintptr_t ad = reinterpret_cast<uintptr_t>(p);
  if (kAligned || (c + 8 <= cols && (ad & 15) == 0)) {
#pragma unroll
    for (int g = 0; g < NG; ++g)
      reinterpret_cast<uint4*>(p)[g] = make_uint4(r.w[4 * g], r.w[4 * g + 1], r.w[4 * g + 2], r.w[4 * g + 3]);
    return;
  }
  if constexpr (!kAligned) {
    if (c + 8 > cols) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (c + i < cols) {
          if constexpr (kB == 2) reinterpret_cast<uint16_t*>(p)[i] = uint16_t(r.w[i >> 1] >> (16 * (i & 1)));
          else reinterpret_cast<uint32_t*>(p)[i] = r.w[i];
        }
      }
    } else if (kB == 4 || (ad & 3) == 0) {
#pragma unroll
      for (int i = 0; i < NW; ++i) reinterpret_cast<uint32_t*>(p)[i] = r.w[i];
    } else {
      reinterpret_cast<uint16_t*>(p)[0] = uint16_t(r.w[0]);
#pragma unroll
      for (int i = 0; i + 1 < NW; ++i)
        *reinterpret_cast<uint32_t*>(p + 2 + 4 * i) = __funnelshift_r(r.w[i], r.w[i + 1], 16);
      *reinterpret_cast<uint16_t*>(p + 14) = uint16_t(r.w[NW - 1] >> 16);
    }
  }
}

// Eight code bytes (lo, hi) to columns c .. c+7 of a code row.
template <bool kAligned>
__device__ __forceinline__ void store8_codes(uint8_t* row, int c, int cols, uint32_t lo, uint32_t hi) {
  if (c >= cols) return;
  if constexpr (kAligned) {
    *reinterpret_cast<uint2*>(row + c) = make_uint2(lo, hi);
  } else if (c + 8 <= cols) {
    store8_any(row + c, lo, hi);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < cols) row[c + i] = uint8_t((i < 4 ? lo : hi) >> (8 * (i & 3)));
  }
}

}  // namespace fp8ds
