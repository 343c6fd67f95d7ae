// What fp16 takes from the gradients' left operand, and its way back.
//
// A row of the left operand is dY * scale times a power of two that puts its largest value at
// 2^13..2^14. A value below 2^-14, that is below 2^-27 of the largest, has no normal fp16 and loses
// up to 2^-25, all of itself where that is less. Beside larger terms that is nothing, but int8
// operands hold many zeros: where all larger terms meet one, a result rests on what was lost.
//
// So whoever rounds a row adds up what its values lose, L. A result's sum is off by no more than
// 128 L for it; if the sum is at least 2^18 L, that is within 2^-11 of it, a rounding of fp16 more,
// and it stands. Otherwise, unless its column of the int8 operand holds nothing but zeros, its row
// is multiplied once more: the lost parts, as bf16 numbers (8 bits, fp32's range), are a second left
// operand, and the tile (or the workgroup of a gradient of few rows) goes over the contraction
// again with those rows of it, the others zero. A lost part that counts is within 2^-8 of itself,
// down to 2^-139 of its row's largest, where the scaled value leaves fp32's normal range.
//
// Which rows those are depends on the row itself and the int8 operand, so rows stay independent of
// one another, and no data take more than the contraction twice.
//
// Rows whose values lie near one another pay for the search alone, old and new in us: 2048 rows of
// 4096 x 11008 193.5 and 195.4 (input), 205.4 and 209.8 (weights), 150 rows of 11008 x 4096 29.7 and
// 30.1, 777 rows of 5120 x 1536 26.2 and 27.2, rank 16 of 1999 rows 9.6 and 10.1; channels of zeros
// cost nothing more. One token 2^40 above the rest: weights of 4096 x 11008 over 2048 rows 171 and
// 421, 5120 x 1536 over 777 26.0 and 58.2. Gradients of a softmax over 32000 channels, 2048 rows of
// 4096, whose values cover hundreds of binades (logits of standard deviation 5 and 9): input 554 and
// 1011, 480 and 930, weights 573 and 965, 517 and 977. Mended one result at a time by a wave, the
// softmaxes took less (951, 1466, 623, 596), but what one token or channels of zeros can put at risk
// up to seconds.
#pragma once

#include "i8_device.hpp"

namespace q4 {

constexpr float kLeast16 = 0x1p-14f;  // fp16's least normal number
constexpr float kLostUnit = 0x1p-29f;
constexpr float kLostLimit = 0x1p18f;

// The least magnitude of values that are not zero, as 2 * its bits - 1: zeros become the largest
// number by themselves. It tells in one and a half instructions a value whether a lane has
// anything to add up, which takes five.
constexpr uint32_t kNoLeast = 0xffffffffu;
__device__ __forceinline__ uint32_t least_of(uint32_t least, float x) {
  return min(least, (__builtin_bit_cast(uint32_t, x) << 1) - 1u);
}
__device__ __forceinline__ float scaled_least(uint32_t least, float up) {
  return __builtin_bit_cast(float, least >> 1) * up;  // of no values: a NaN
}
__device__ __forceinline__ bool may_lose(uint32_t least, float up) {
  return scaled_least(least, up) < kLeast16;
}

// what v loses as fp16; exact
__device__ __forceinline__ float lost16(float v) {
  return fabsf(v) < kLeast16 ? v - (float)(_Float16)v : 0.0f;
}
// the same as a bf16 number, to nearest (it is finite)
__device__ __forceinline__ uint32_t lost_bf16(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, lost16(v));
  return (u + 0x7fffu + ((u >> 16) & 1u)) >> 16;
}
// Sums over lanes are kept in whole units, rounded up: added in any order they are the same. At most
// 16 units a value, and fewer than 2^27 values a row.
__device__ __forceinline__ void add_lost(uint32_t* units, float lost) {
  if (lost > 0.0f) atomicAdd(units, (uint32_t)ceilf(lost * (1.0f / kLostUnit)));
}
// a sum below this does not stand
__device__ __forceinline__ float lost_limit(uint32_t units) {
  return (float)units * (kLostUnit * kLostLimit);
}

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
// Eight int8 as bf16 numbers, exactly.
__device__ __forceinline__ bf16x8 to_bf16s(int2v q) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = (uint32_t)q[i / 2] >> (16 * (i % 2));
    const float lo = (float)(int8_t)w, hi = (float)(int8_t)(w >> 8);
    h[i] = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, hi), __builtin_bit_cast(uint32_t, lo),
                                 0x07060302u);
  }
  return __builtin_bit_cast(bf16x8, make_uint4(h[0], h[1], h[2], h[3]));
}

}  // namespace q4
