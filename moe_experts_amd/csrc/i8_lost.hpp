// What fp16 takes from the gradients' left operand, and its way back.
//
// A row of the left operand is dY * scale times a power of two that puts its largest value at
// 2^13..2^14. A value below 2^-14, that is below 2^-27 of the largest, has no normal fp16 and loses
// up to 2^-25, all of itself where that is less. Beside larger terms that is nothing, but int8
// operands hold many zeros: where all larger terms meet one, a result rests on what was lost.
//
// So whoever rounds a row adds up what its values lose, L. A result's sum is off by no more than
// 128 L for it. If its terms' magnitudes add up to 2^18 L, that is within 2^-11 of them, as much as
// the rounding of every term to fp16 is, and it stands. The sum itself tells that of nearly all
// results. For any other a wave adds up its terms' magnitudes, which in a few steps is enough for
// nearly all of these, and else the lost parts' products, from dY in fp32. Which results those are
// depends on their own row and column alone, so rows stay independent of one another. Splits of
// tiles are mended where they are added; splits of few rows, which are scaled each by itself, each
// by itself. Terms down to 2^-139 of a row's largest count, where the scaled value leaves fp32's
// normal range.
//
// Rows whose values lie near one another pay for the search alone: 150 rows of 11008 x 4096 29.3 ->
// 29.8 us, rank 16 of 1999 rows 9.5 -> 9.9, 777 rows of 5120 x 1536 25.8 -> 26.4, 2048 of 4096 x
// 11008 202 -> 203 (input) and 212 -> 214 (weights). Gradients of a softmax over 32000 channels,
// 2048 rows of 4096, whose values cover hundreds of binades (logits of standard deviation 5 and 9):
// input 583 -> 959 and 527 -> 1475 us, weights 603 -> 639 and 531 -> 604; with one channel of 20
// dead 596 -> 1106. Added instead to all results of a block of 32 x 32 with one to mend, by the
// matrix cores and without the early end, the same took 1240 to 10400.
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

// what v loses as fp16
__device__ __forceinline__ float lost16(float v) {
  return fabsf(v) < kLeast16 ? v - (float)(_Float16)v : 0.0f;
}
// Sums over lanes are kept in whole units, rounded up: added in any order they are the same. At most
// 16 units a value, and fewer than 2^27 values a row.
__device__ __forceinline__ void add_lost(uint32_t* units, float lost) {
  if (lost > 0.0f) atomicAdd(units, (uint32_t)ceilf(lost * (1.0f / kLostUnit)));
}
// below this a result's sum is mended
__device__ __forceinline__ float lost_limit(uint32_t units) {
  return (float)units * (kLostUnit * kLostLimit);
}

// Which of R columns of B from col0 on are not all zeros from c0 to c1, a bit each, among those that
// are wanted; the same for all lanes of the wave. Columns that hold nothing (dead channels) would
// otherwise be searched to their end for every row.
template <int R>
__device__ __forceinline__ uint32_t live_columns(const LeftSource& s, int col0, uint32_t wanted,
                                                 int c0, int c1) {
  constexpr int kPieces = R / 16, kPlaces = kWaveSize / kPieces;  // of a load
  const int lane = threadIdx.x & 63, piece = 16 * (lane % kPieces);
  uint32_t live = 0;
#pragma unroll 1
  for (int c = c0; c < c1 && (wanted & ~live) != 0; c += 8 * kPlaces) {
    uint32_t any[4] = {};
    if (col0 + piece < s.cols)
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int at = min(c + u * kPlaces + lane / kPieces, c1 - 1);
        uint32_t w[4];
        __builtin_memcpy(w, __builtin_assume_aligned(s.B + (size_t)at * s.cols + col0 + piece, 16), 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) any[i] |= w[i];
      }
    uint32_t bits = 0;
#pragma unroll
    for (int e = 0; e < 16; ++e) bits |= (any[e / 4] >> (8 * (e % 4)) & 255u) != 0 ? 1u << e : 0u;
    bits <<= piece;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) bits |= (uint32_t)__shfl_xor((int)bits, o);
    live |= bits;
  }
  return __builtin_amdgcn_readfirstlane(live & wanted);
}

// Sum of the products of what a row, scaled by `up`, lost from c0 to c1, or 0 as soon as its terms'
// magnitudes have reached `limit`. Row and column are the same for all lanes of the wave, and so is
// the result.
__device__ __forceinline__ float lost_sum(const LeftSource& s, int row, float up, float limit,
                                          int col, int c0, int c1) {
  float sum = 0.0f, size = 0.0f;
  const uint16_t* y = s.dY + (size_t)row * s.row_step;
#pragma unroll 1
  for (int c = c0; c < c1; c += 4 * kWaveSize) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int place = c + u * kWaveSize + (int)(threadIdx.x & 63);
      const size_t at = min(place, c1 - 1);
      const float v = Val<Q4_TYPE_BF16>::get(y[at * s.step]) * s.scale[at] * up;
      const float q = place < c1 ? (float)s.B[at * s.cols + col] : 0.0f;
      size += fabsf(v * q);
      sum += lost16(v) * q;
    }
    if (__any(size >= limit)) return 0.0f;
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
  return sum;
}

// Mends a wave's MI x NJ blocks of R x R results as the matrix instructions of R rows leave them:
// lane l holds row row0 + R * i + l % R, register r of block j column col0 + R * j + 8 * (r / 4) +
// 4 * (l / R) + r % 4. limit and up are the rows', limit 0 for one that is not to be touched. One
// copy of the loop serves all blocks: the tiles have no registers for more.
template <int R, int MI, int NJ, class V>
__device__ __forceinline__ void mend_lost(V (&acc)[MI][NJ], const LeftSource& s, int row0, int col0,
                                          int c0, int c1, const float (&limit)[MI],
                                          const float (&up)[MI]) {
  constexpr int kRegs = R * R / kWaveSize;
  const int lane = threadIdx.x & 63;
  uint32_t low[MI * NJ];
  uint32_t any = 0;
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      uint32_t bits = 0;
#pragma unroll
      for (int r = 0; r < kRegs; ++r)
        if (col0 + R * j + 8 * (r / 4) + 4 * (lane / R) + r % 4 < s.cols &&
            fabsf(acc[i][j][r]) < limit[i])
          bits |= 1u << r;
      low[i * NJ + j] = bits;
      any |= bits;
    }
  if (!__any(any)) return;
#pragma unroll 1
  for (int block = 0; block < MI * NJ; ++block) {
    uint32_t bits = low[0];
    float block_limit = limit[0], block_up = up[0];
#pragma unroll
    for (int b = 1; b < MI * NJ; ++b)
      if (block == b) {
        bits = low[b];
        block_limit = limit[b / NJ];
        block_up = up[b / NJ];
      }
    // lanes with a result to look at in column `in`, in register `reg`
    auto rows_of = [&](int in, int& reg) {
      reg = R == 32 ? in / 8 * 4 + in % 4 : in % 4;
      return __ballot((bits >> reg & 1u) && lane / R == (R == 32 ? in / 4 % 2 : in / 4));
    };
    const int first = col0 + block % NJ * R;
    int reg;
    uint32_t wanted = 0;
#pragma unroll 1
    for (int in = 0; in < R; ++in) wanted |= rows_of(in, reg) != 0 ? 1u << in : 0u;
    if (wanted != 0) wanted = live_columns<R>(s, first, wanted, c0, c1);
#pragma unroll 1
    for (; wanted != 0; wanted &= wanted - 1) {
      const int in = __builtin_ctz(wanted);
#pragma unroll 1
      for (uint64_t rows = rows_of(in, reg); rows != 0; rows &= rows - 1) {
        const int l = __builtin_ctzll(rows);
        auto of_row = [&](float f) {
          return __builtin_bit_cast(float,
                                    __builtin_amdgcn_readlane(__builtin_bit_cast(int, f), l));
        };
        const float sum = lost_sum(s, row0 + block / NJ * R + l % R, of_row(block_up),
                                   of_row(block_limit), first + in, c0, c1);
#pragma unroll
        for (int b = 0; b < MI * NJ; ++b)
#pragma unroll
          for (int r = 0; r < kRegs; ++r) {
            const float v = acc[b / NJ][b % NJ][r];
            acc[b / NJ][b % NJ][r] = lane == l && b == block && r == reg ? v + sum : v;
          }
      }
    }
  }
}

}  // namespace q4
