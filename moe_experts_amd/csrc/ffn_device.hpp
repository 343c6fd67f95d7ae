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

#include "ffn_internal.hpp"
#include "q4_device.hpp"
#include "q4moe.h"

namespace q4 {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef float float4v __attribute__((ext_vector_type(4)));

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

// ---------------------------------------------------------------------------
// Adapters, narrow half, few rows: one wave per (row m, rank index r) runs one
// dot product of K, eight values a lane and step; the lanes are added by a
// fixed butterfly. Every adapter row is read once for every row of x that uses
// it (16-byte loads), so this form is for rows that mostly use different
// adapters. A row without adapter gets zeros.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4v a = *reinterpret_cast<const float4v*>(p);
  const float4v b = *reinterpret_cast<const float4v*>(p + 4);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[e] = a[e];
    v[4 + e] = b[e];
  }
}
__device__ __forceinline__ void load8(const _Float16* p, float (&v)[8]) {
  const half8 a = *reinterpret_cast<const half8*>(p);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = (float)a[e];
}

template <class X>
__device__ __forceinline__ void shrink_wave(const X* __restrict__ x, const Adapters& ad,
                                            float* __restrict__ t, int M, int K, int w) {
  const int lane = threadIdx.x & 63;
  const int m = w / ad.R;
  if (m >= M) return;
  const int r = w - m * ad.R;
  const int id = ad.ids[m];
  float sum = 0.0f;
  if (id >= 0 && id < ad.L) {
    const X* xr = x + (size_t)m * K;
    const _Float16* ar = reinterpret_cast<const _Float16*>(ad.A) + ((size_t)id * ad.R + r) * K;
    constexpr int kStep = 64 * 8, kUnroll = 4;
    for (int k0 = lane * 8; k0 < K; k0 += kStep * kUnroll) {
      float xv[kUnroll][8], av[kUnroll][8];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        // past the end the last group is read again and not added
        const int k = min(k0 + u * kStep, K - 8);
        load8(xr + k, xv[u]);
        load8(ar + k, av[u]);
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (k0 + u * kStep < K)
#pragma unroll
          for (int e = 0; e < 8; ++e) sum = __builtin_fmaf(xv[u][e], av[u][e], sum);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
    sum *= ad.scale[id];
  }
  if (lane == 0) t[(size_t)m * ad.R + r] = sum;
}

}  // namespace q4
