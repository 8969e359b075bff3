// Activations of the product's epilogue and their slopes, in float32.
//
//   relu  max(z, 0)                       slope 0 for z <= 0, else 1
//   silu  z p,  p = 1 / (1 + e^-z)        slope p + z p q,  q = 1 - p
//   gelu  z p,  p = 1 / (1 + e^-w),       slope p + z p q w'
//         w = 2 sqrt(2/pi) (z + 0.044715 z^3): the tanh form, since
//         (1 + tanh(w/2)) / 2 is the logistic function of w
//
// Everywhere from e^-w and one reciprocal, two values at a time: the tile
// kernels' epilogue warps have some 20 issue slots per element while the next
// tile's products run, so each operation that can is a packed one.  e^-w grows
// without bound for w << 0: its sum's reciprocal is then 0, and so is the value.
// One formula for every kernel, so that a row's result from one z does not depend
// on how many rows there are.  The fast exponential (2 ulp, and |w| times the
// rounding of its argument) and reciprocal (1 ulp) are far inside what the 8- and
// 16-bit outputs keep.
#pragma once

#include "common.cuh"
#include "fp8_ring.cuh"
#include "fp8ds_layer.h"

namespace fp8ds {

constexpr float kGeluC2 = 1.5957691216057308f;  // 2 sqrt(2/pi)
constexpr float kGeluA = 0.044715f;

// z^2, kept finite so that 0 * z^2 stays 0 where p q has vanished.
__device__ __forceinline__ float square_capped(float z) { return fminf(z * z, 1.0e30f); }

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float rcp_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

constexpr float kLog2E = 1.4426950408889634f;

template <int ACT>
__device__ __forceinline__ void act_pair(float& a, float& b) {
  if constexpr (ACT == FP8_ACT_RELU) {
    a = max_nan(a, 0.0f);
    b = max_nan(b, 0.0f);
  } else {
    float x = a, y = b;  // -> e^-w + 1
    if constexpr (ACT == FP8_ACT_GELU) {
      constexpr float c1 = -kGeluC2 * kLog2E;
      mul2(x, y, a, b);
      fma2(x, y, c1 * kGeluA, c1, c1);
      mul2(x, y, a, b);
    } else {
      scale2(x, y, -kLog2E);
    }
    x = exp2_fast(x);
    y = exp2_fast(y);
    add2(x, y, 1.0f, 1.0f);
    mul2(a, b, rcp_fast(x), rcp_fast(y));
  }
}

// act of one value.
__device__ __forceinline__ float act_one(int act, float z) {
  float y = z, same = z;
  switch (act) {
    case FP8_ACT_RELU: act_pair<FP8_ACT_RELU>(y, same); break;
    case FP8_ACT_GELU: act_pair<FP8_ACT_GELU>(y, same); break;
    case FP8_ACT_SILU: act_pair<FP8_ACT_SILU>(y, same); break;
    default: break;
  }
  return y;
}

// value and slope of a pair: q = 1 - p is off by at most 2^-24, which the slope
// p + z p q multiplies by |z p|.  z^2 is capped so that p q = 0 times it is 0.
template <int ACT>
__device__ __forceinline__ void act_slope_pair(float& a, float& b, float& sa, float& sb) {
  if constexpr (ACT == FP8_ACT_NONE) {
    sa = sb = 1.0f;
  } else if constexpr (ACT == FP8_ACT_RELU) {
    sa = a <= 0.0f ? 0.0f : 1.0f;
    sb = b <= 0.0f ? 0.0f : 1.0f;
    a = max_nan(a, 0.0f);
    b = max_nan(b, 0.0f);
  } else {
    float x = a, y = b, wx = 1.0f, wy = 1.0f;  // e^-w; w'
    if constexpr (ACT == FP8_ACT_GELU) {
      constexpr float c1 = -kGeluC2 * kLog2E;
      const float s = square_capped(a), t = square_capped(b);
      x = s, y = t;
      fma2(x, y, c1 * kGeluA, c1, c1);
      mul2(x, y, a, b);
      wx = s, wy = t;
      fma2(wx, wy, 3.0f * kGeluC2 * kGeluA, kGeluC2, kGeluC2);
    } else {
      scale2(x, y, -kLog2E);
    }
    x = exp2_fast(x);
    y = exp2_fast(y);
    add2(x, y, 1.0f, 1.0f);
    const float p = rcp_fast(x), r = rcp_fast(y);
    mul2(a, b, p, r);
    sa = p, sb = r;
    fma2(sa, sb, -1.0f, 1.0f, 1.0f);  // q
    if constexpr (ACT == FP8_ACT_GELU) mul2(sa, sb, wx, wy);
    fma2v(sa, sb, a, b, p, r);
  }
}

}  // namespace fp8ds
