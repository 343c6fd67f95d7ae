// Device-side pieces of the dense feed-forward kernels.
//
// Activations of the gated block and their slopes, in fp32.
//   SiLU:  a(z) = z * s(z),        a'(z) = s + z * s * (1 - s)
//   GELU (tanh form): a(z) = z * s(p), p = 2c (z + 0.044715 z^3), c = sqrt(2/pi),
//          since (1 + tanh v) / 2 = s(2v);  a'(z) = s + z * s * (1 - s) * p'(z)
// with s(v) = 1 / (1 + exp(-v)). For v below about -88 exp overflows to
// infinity and s is exactly 0; z = -inf gives -inf * 0 = NaN as the formula does.
#pragma once

#include <hip/hip_runtime.h>

#include "q4moe.h"

namespace q4 {

__device__ __forceinline__ float sigmoid_f(float v) { return 1.0f / (1.0f + expf(-v)); }

__device__ __forceinline__ float act_arg(float z, int act) {
  constexpr float c2 = 1.5957691216057308f;  // 2 * sqrt(2 / pi)
  return act == Q4_ACT_SILU ? z : c2 * (z + 0.044715f * z * z * z);
}

__device__ __forceinline__ float act_value(float z, int act) {
  return z * sigmoid_f(act_arg(z, act));
}

__device__ __forceinline__ void act_value_slope(float z, int act, float& a, float& slope) {
  constexpr float c2 = 1.5957691216057308f;
  const float s = sigmoid_f(act_arg(z, act));
  // s * (1 - s) from s alone: for s near 1 the difference is exact in fp32
  const float dp = act == Q4_ACT_SILU ? 1.0f : c2 * (1.0f + 0.134145f * z * z);
  a = z * s;
  slope = s + z * (s * (1.0f - s)) * dp;
}

}  // namespace q4
