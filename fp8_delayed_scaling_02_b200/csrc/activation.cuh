// Activations of the product's epilogue and their slopes, in float32.
//
//   relu  max(z, 0)                       slope z > 0
//   silu  z p,  p = 1 / (1 + e^-z)        slope p + z p q,  q = 1 - p
//   gelu  z p,  p = 1 / (1 + e^-w),       slope p + z p q w'
//         w = 2 sqrt(2/pi) (z + 0.044715 z^3): the tanh form, since
//         (1 + tanh(w/2)) / 2 is the logistic function of w
//
// p and q both come from t = e^-|w| in (0, 1]: r = 1/(1+t) is one of them and
// t r the other, so neither cancels nor overflows, however large |w|.  The
// fast exponential and division are within (2 + 1.2 |w|) and 2 float32 ulp
// (CUDA's stated bounds): far inside what the 8- and 16-bit outputs keep.
#pragma once

#include "common.cuh"
#include "fp8ds_layer.h"

namespace fp8ds {

constexpr float kGeluC2 = 1.5957691216057308f;  // 2 sqrt(2/pi)
constexpr float kGeluA = 0.044715f;

__device__ __forceinline__ void logistic(float w, float& p, float& q) {
  const float t = __expf(-fabsf(w));
  const float r = __fdividef(1.0f, 1.0f + t);
  const float tr = t * r;
  p = w >= 0.0f ? r : tr;
  q = w >= 0.0f ? tr : r;
  if (w != w) p = w;
}

// z^2, kept finite so that 0 * z^2 stays 0 where p q has vanished.
__device__ __forceinline__ float square_capped(float z) { return fminf(z * z, 1.0e30f); }

__device__ __forceinline__ float act_value(int act, float z) {
  float p, q;
  switch (act) {
    case FP8_ACT_RELU: return z < 0.0f ? 0.0f : z;  // NaN stays NaN
    case FP8_ACT_SILU: logistic(z, p, q); return z * p;
    case FP8_ACT_GELU: logistic(z * fmaf(kGeluC2 * kGeluA, square_capped(z), kGeluC2), p, q); return z * p;
    default: return z;
  }
}

__device__ __forceinline__ void act_value_slope(int act, float z, float& value, float& slope) {
  float p, q;
  switch (act) {
    case FP8_ACT_RELU:
      value = z < 0.0f ? 0.0f : z;
      slope = z > 0.0f ? 1.0f : 0.0f;
      return;
    case FP8_ACT_SILU:
      logistic(z, p, q);
      value = z * p;
      slope = fmaf(value, q, p);
      return;
    case FP8_ACT_GELU: {
      const float s = square_capped(z);
      logistic(z * fmaf(kGeluC2 * kGeluA, s, kGeluC2), p, q);
      value = z * p;
      slope = fmaf(value * q, fmaf(3.0f * kGeluC2 * kGeluA, s, kGeluC2), p);
      return;
    }
    default:
      value = z;
      slope = 1.0f;
  }
}

}  // namespace fp8ds
