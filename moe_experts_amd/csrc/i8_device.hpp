// Device-side pieces of the 8-bit kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "i8_internal.hpp"
#include "q4_device.hpp"
#include "q4moe.h"

namespace q4 {

typedef int int4v __attribute__((ext_vector_type(4)));
typedef int int2v __attribute__((ext_vector_type(2)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef float float4v __attribute__((ext_vector_type(4)));
typedef int int16v __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void lds_void_t;

// fp32 -> bf16, to nearest, ties to even; a NaN stays one.
__device__ __forceinline__ uint32_t i8_to_bf16(float f) {
  const uint32_t u = __builtin_bit_cast(uint32_t, f);
  if ((u & 0x7fffffffu) > 0x7f800000u) return (u >> 16) | 0x40u;
  return (u + 0x7fffu + ((u >> 16) & 1u)) >> 16;
}

// Types of results and activations: bytes, and conversions from and to fp32.
template <int TYPE>
struct Val;
template <>
struct Val<Q4_TYPE_F32> {
  typedef float T;
  static __device__ __forceinline__ float get(T v) { return v; }
  static __device__ __forceinline__ T put(float f) { return f; }
};
template <>
struct Val<Q4_TYPE_F16> {
  typedef _Float16 T;
  static __device__ __forceinline__ float get(T v) { return (float)v; }
  static __device__ __forceinline__ T put(float f) { return (_Float16)f; }
};
template <>
struct Val<Q4_TYPE_BF16> {
  typedef uint16_t T;
  static __device__ __forceinline__ float get(T v) {
    return __builtin_bit_cast(float, (uint32_t)v << 16);
  }
  static __device__ __forceinline__ T put(float f) { return (uint16_t)i8_to_bf16(f); }
};

// Runs `call` with the type as a compile-time number.
template <class F>
void i8_by_type(int type, F&& call) {
  if (type == Q4_TYPE_F32)
    call(std::integral_constant<int, Q4_TYPE_F32>{});
  else if (type == Q4_TYPE_F16)
    call(std::integral_constant<int, Q4_TYPE_F16>{});
  else
    call(std::integral_constant<int, Q4_TYPE_BF16>{});
}

// ---------------------------------------------------------------------------
// Rows to int8. The scale of a row is s = max|x| / 127 rounded to fp32, and q the
// whole number nearest to the real quotient x / s, ties to even. In fp32 the
// quotient x * (1 / s) is rounded, and a value close to a half may go the wrong way
// by that; but the remainder r = x - q * s of a candidate q at most one off is an
// fp32 number (x and q * s are multiples of s's last place, or x itself is small),
// so the fused multiply-add gives it exactly, and comparing it with s / 2 decides.
// Scales below 2^-64 are worked with times 2^64, both in x and s, which is exact, so
// that neither 1 / s nor r leaves the normal range.
// ---------------------------------------------------------------------------
struct RowScale {
  float s;     // as stored
  float f;     // what x is multiplied by first: 1 or 2^64
  float sf;    // s * f
  float inv;   // 1 / sf, 0 for a row that becomes all zeros
};

// big: the largest bit pattern of |x| in the row. A row with an infinity or a NaN gets a
// NaN for its scale, and zeros.
__device__ __forceinline__ RowScale row_scale(uint32_t big) {
  RowScale r;
  const float amax = __builtin_bit_cast(float, big);
  const bool bad = big >= 0x7f800000u;
  r.s = bad ? __builtin_bit_cast(float, 0x7fc00000u) : amax / 127.0f;
  r.f = r.s < 0x1p-64f ? 0x1p64f : 1.0f;
  r.sf = r.s * r.f;
  r.inv = bad || r.s == 0.0f ? 0.0f : 1.0f / r.sf;
  return r;
}

__device__ __forceinline__ uint32_t magnitude(float x) {
  return __builtin_bit_cast(uint32_t, x) & 0x7fffffffu;
}

// N values (a multiple of 4) to N int8 in N / 4 dwords.
template <int N>
__device__ __forceinline__ void to_int8(const float (&x)[N], const RowScale& rs,
                                        uint32_t (&out)[N / 4]) {
  constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: the low bits of t are q in two's complement
  if (rs.inv == 0.0f) {                  // uniform in a row
#pragma unroll
    for (int i = 0; i < N / 4; ++i) out[i] = 0;
    return;
  }
  float t[N];
  float far = 0.0f;
  const float half = 0.5f * rs.sf;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float v = x[i] * rs.f;
    t[i] = __builtin_fmaf(v, rs.inv, kMagic);
    far = fmaxf(far, fabsf(__builtin_fmaf(kMagic - t[i], rs.sf, v)));
  }
  // a tie, a candidate next to a half, or (subnormal scales) quotients past 127
  if (far >= half || rs.s < 0x1p-126f) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float v = x[i] * rs.f;
      const float q = t[i] - kMagic;
      const float r = __builtin_fmaf(-q, rs.sf, v);
      const bool odd = __builtin_bit_cast(uint32_t, t[i]) & 1u;
      const bool away = fabsf(r) > half || (fabsf(r) == half && odd);
      float c = away ? q + copysignf(1.0f, r) : q;
      c = fminf(fmaxf(c, -127.0f), 127.0f);
      t[i] = c + kMagic;
    }
  }
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const uint32_t a = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, t[4 * i + 1]),
                                             __builtin_bit_cast(uint32_t, t[4 * i]), 0x0c0c0400u);
    const uint32_t b = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, t[4 * i + 3]),
                                             __builtin_bit_cast(uint32_t, t[4 * i + 2]),
                                             0x04000c0cu);
    out[i] = a | b;
  }
}

// A barrier for LDS alone: copies from memory stay in flight over it.
__device__ __forceinline__ void lds_only_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Largest of a workgroup's values; every lane gets it. `at`: LDS of one dword a wave.
template <int THREADS>
__device__ __forceinline__ uint32_t workgroup_max(uint32_t v, uint32_t* at) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o));
  if constexpr (THREADS > kWaveSize) {
    if ((threadIdx.x & 63) == 0) at[threadIdx.x >> 6] = v;
    __syncthreads();
    v = at[0];
#pragma unroll
    for (int w = 1; w < THREADS / kWaveSize; ++w) v = max(v, at[w]);
  }
  return v;
}

// The largest of a wave's values of eight columns, dealt out to the lanes while they are
// reduced: with lanes a multiple of STRIDE apart holding values of the same columns, lanes
// below 8 * STRIDE end with a column each in v[0], the one that is returned.
template <int STRIDE>
__device__ __forceinline__ int wave_max_of_eight(uint32_t (&v)[8]) {
  const int lane = threadIdx.x & 63;
  int e = 0;
#pragma unroll
  for (int half = 4, o = STRIDE; half > 0; half >>= 1, o <<= 1) {
    const bool up = lane & o;
    e += up ? half : 0;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const uint32_t keep = up ? v[i + half] : v[i], send = up ? v[i] : v[i + half];
      v[i] = max(keep, (uint32_t)__shfl_xor((int)send, o));
    }
  }
#pragma unroll
  for (int o = 8 * STRIDE; o < kWaveSize; o <<= 1)
    v[0] = max(v[0], (uint32_t)__shfl_xor((int)v[0], o));
  return e;
}

// Eight values as they stand in memory (aligned to one value). Kept so, 16-bit types take half
// the registers.
template <int TYPE>
struct Piece {
  typedef typename Val<TYPE>::T T;
  static constexpr int kWords = sizeof(T) * 2;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* __restrict__ p) { __builtin_memcpy(w, p, sizeof(w)); }
  // Keeps the compiler from holding the values converted from one use to the next.
  __device__ __forceinline__ void fresh() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) asm volatile("" : "+v"(w[i]));
  }
  __device__ __forceinline__ float operator[](int e) const {
    if constexpr (sizeof(T) == 4)
      return __builtin_bit_cast(float, w[e]);
    else if constexpr (TYPE == Q4_TYPE_BF16)
      return __builtin_bit_cast(float, e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
    else
      return (float)__builtin_bit_cast(_Float16, (uint16_t)(w[e / 2] >> (16 * (e & 1))));
  }
};

// ---------------------------------------------------------------------------
// Left operands of the gradients. A product dY * scale is rounded to fp16 once: within 2^-11 of
// itself, where bf16 would be within 2^-8, as much as the result's own rounding; it adds 0.6 to
// 1.2 % to the error that the result has by that. Gradients lie far below fp16's range, so the
// values that one sum adds are scaled together by a power of two (exact) that takes the largest of
// them to 2^13..2^14; the sum is scaled back. What becomes of those that are still too small is in
// i8_lost.hpp.
// ---------------------------------------------------------------------------
struct PowerOfTwo {
  float up, down;
};
__device__ __forceinline__ PowerOfTwo to_fp16_range(uint32_t big) {
  // zeros, infinities and NaN stay as they are
  const bool plain = big == 0 || big >= 0x7f800000u;
  const int e = plain ? 0 : min(126, 13 + 127 - (int)(big >> 23));
  PowerOfTwo p;
  p.up = __builtin_bit_cast(float, (uint32_t)(127 + e) << 23);
  p.down = __builtin_bit_cast(float, (uint32_t)(127 - e) << 23);
  return p;
}

// Eight int8 as halves, exactly: with the sign bit turned, a byte behind 0x64 is the half
// 1024 + 128 + q.
__device__ __forceinline__ half8 to_halves(int2v q) {
  uint32_t h[4];
  const half2v off = {(_Float16)1152.0f, (_Float16)1152.0f};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t u = (uint32_t)q[i] ^ 0x80808080u;
    h[2 * i] = __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u);
    h[2 * i + 1] = __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h[i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2v, h[i]) - off);
  return __builtin_bit_cast(half8, make_uint4(h[0], h[1], h[2], h[3]));
}

}  // namespace q4
