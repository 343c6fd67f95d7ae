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

// FAST takes the hardware's exp2 and reciprocal (each within about 1 ulp) instead
// of expf and a division: s is then off by at most about (|v| + 4) * 2^-24 of
// itself, which disappears in a result rounded to fp16 (2^-11), at a third of the
// instructions.
template <bool FAST>
__device__ __forceinline__ float sigmoid_f(float v) {
  if constexpr (FAST)
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504088896341f * v));
  else
    return 1.0f / (1.0f + expf(-v));
}

__device__ __forceinline__ float act_arg(float z, int act) {
  constexpr float c2 = 1.5957691216057308f;  // 2 * sqrt(2 / pi)
  return act == Q4_ACT_SILU ? z : c2 * (z + 0.044715f * z * z * z);
}

template <bool FAST>
__device__ __forceinline__ float act_value(float z, int act) {
  return z * sigmoid_f<FAST>(act_arg(z, act));
}

// value and slope of a gate, for results of 16 bits
__device__ __forceinline__ void act_value_slope(float z, int act, float& a, float& slope) {
  constexpr float c2 = 1.5957691216057308f;
  const float s = sigmoid_f<true>(act_arg(z, act));
  const float dp = act == Q4_ACT_SILU ? 1.0f : c2 * (1.0f + 0.134145f * z * z);
  a = z * s;
  slope = s + z * (s * (1.0f - s)) * dp;
}

// fp32 -> bf16, to nearest, ties to even; a NaN stays one (its high bits with
// the quiet bit set).
__device__ __forceinline__ uint16_t float_to_bf16(float f) {
  const uint32_t u = __builtin_bit_cast(uint32_t, f);
  if ((u & 0x7fffffffu) > 0x7f800000u) return (uint16_t)((u >> 16) | 0x40u);
  return (uint16_t)((u + 0x7fffu + ((u >> 16) & 1u)) >> 16);
}

}  // namespace q4
