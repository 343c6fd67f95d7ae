// Pieces of the 8-bit operators' GEMM tiles: copies of a K step into LDS, the hand-over
// between steps and the way results leave.
//
// A step holds 128 bytes of each row of the left operand (128 int8 or 64 fp16), copied
// memory -> LDS without passing through registers (16 bytes a lane, eight lanes a row). The
// 16-byte chunk c of row r stands at chunk c ^ swz(r): a copy writes LDS in lane order, so
// the lane asks for the chunk that belongs at its place. Sixteen rows that a matrix operand
// reads at once then meet no bank twice.
#pragma once

#include "i8_device.hpp"

namespace q4 {

constexpr uint32_t kPastEnd = 0x80000000u;  // offset past the end of any array
constexpr int kStepBytes = 128;             // of a row of the left operand in a step

// What the chunks of a row are turned by.
__device__ __forceinline__ int swz_row(int r) { return (r >> 1) & 7; }

__device__ __forceinline__ void copy16(__amdgpu_buffer_rsrc_t r, uint8_t* lds, uint32_t off,
                                       uint32_t so) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_t*)lds, 16, off, so, 0, 0);
}

// The copies of ROWS rows of a step by THREADS lanes.
template <int ROWS, int THREADS>
struct RowCopy {
  static constexpr int kChunks = kStepBytes / 16;
  static constexpr int kInstr = ROWS * kChunks / THREADS;
  static_assert(ROWS * kChunks % THREADS == 0 && THREADS / kChunks % 16 == 0,
                "whole copies, one swizzle a lane");
  __amdgpu_buffer_rsrc_t r;
  uint32_t off[kInstr];
  int chunk;  // 16 * (the lane's chunk in a step)
  // `rows` (at least one) rows of `pitch` bytes from `base`; rows past them repeat the last
  __device__ __forceinline__ void init(const void* base, int rows, uint32_t pitch, int t) {
    r = make_rsrc(base, (uint32_t)rows * pitch);
    chunk = 16 * ((t % kChunks) ^ swz_row(t / kChunks));
#pragma unroll
    for (int i = 0; i < kInstr; ++i)
      off[i] = (uint32_t)min((i * THREADS + t) / kChunks, rows - 1) * pitch + (uint32_t)chunk;
  }
  // Step ks into `stage`; bytes past `left` of the step (the row's end) become zeros.
  __device__ __forceinline__ void issue(uint8_t* stage, int ks, int left, int wave) const {
    const uint32_t so = (uint32_t)ks * kStepBytes;
    const bool live = chunk < left;
#pragma unroll
    for (int i = 0; i < kInstr; ++i)
      copy16(r, stage + (i * THREADS + wave * kWaveSize) * 16, live ? off[i] : kPastEnd, so);
  }
};

// Hands LDS over at a barrier: this wave's reads of it are done, and of its copies into it all
// but the last COPIES have landed.
template <int COPIES>
__device__ __forceinline__ void tile_hand_over() {
  static_assert(COPIES < 64, "vmcnt");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  // vmcnt(COPIES) lgkmcnt(0)
  __builtin_amdgcn_s_waitcnt(0x0070 | (COPIES & 15) | (COPIES >> 4) << 14);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Tiles of one pass over the GPU in an order that lets those of an XCD share operands:
// kGroupRows tile rows go down before the next tile column begins.
constexpr int kGroupRows = 8;
__device__ __forceinline__ void tile_of(int L, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int band = kGroupRows * tiles_n;
  const int b = L / band, in = L - b * band;
  const int rows = min(kGroupRows, tiles_m - b * kGroupRows);
  tn = in / rows;
  tm = b * kGroupRows + in - tn * rows;
}

}  // namespace q4
