// 8-bit product of more than 16 rows: Y = (X . W^T) * sx * sw, X int8 [M][K], W int8 [N][K], on
// the integer matrix cores (v_mfma_i32_32x32x32_i8). The sums are whole numbers and exact, so
// splits of the contraction change nothing.
//
// Tiles of BM rows of X and BN rows of W, K steps of 128 bytes. Both operands have their
// contraction contiguous, so a step is copied memory -> LDS as it stands, NS steps in LDS, and a
// lane's 16 bytes of a row are what the matrix instruction takes. One barrier a step.
//   * Large tiles leave the least to move: per 1 KiB of operands that a wave reads from LDS,
//     64 x 96 results give 1.2 products of 32 x 32 x 32, 64 x 64 one, 32 x 32 half of one.
//     256 x 192 is the largest whose accumulators leave room for two sets of operands
//     (256 x 384, one pass of 232 tiles over the CUs: 95 us too, registers spilled).
//   * Small tiles (WHOLE) read all of the next step's operands before they multiply this
//     step's: with 64 to 128 cycles of products a quarter, reading one quarter ahead left
//     them waiting for LDS (130 rows of 4096 x 4096 by 64 x 64: 11.3 -> 9.5 us; 9.8 now).
//
// What bounds it: 2048 rows of 4096 x 11008 take 94 to 105 us, from GPU to GPU, 1.76 to 1.96 POP/s.
// With all CUs busy the power limit holds the clock at 1.69 to 1.72 GHz call after call (2.0 to
// 2.3 in the 777-row product below, which leaves CUs idle), at which the matrix cores' own cycles
// are 52 us; where the whole took 95, it took 85 us without LDS reads, 83 without copies, 72 with
// neither. A deeper ring of
// stages, registers in place of LDS-DMA, raised priorities and freer scheduling all came out
// within 3 %.
//
// Few tiles are bound by the rate at which a CU copies: one workgroup alone on the GPU takes
// 0.25 us a step of 64 x 128, 0.18 of 64 x 64 and 0.31 of 128 x 128, that is 80 cycles a step and
// 21 a KiB (at 64 bytes a cycle it were 16); a fourth stage or other waves over the tile change
// nothing. 777 rows of 5120 x 1536 take 17.5 us of which 40 such steps are 11: 100 CUs have no
// tile, and splits that give them one cost more (22.8 us in two).
#include <algorithm>

#include "i8_device.hpp"
#include "i8_internal.hpp"
#include "i8_tile.hpp"

namespace q4 {
namespace {

struct GemmArgs {
  const int8_t* X;
  const float* sx;
  const int8_t* W;
  const float* sw;
  void* Y;
  int M, N, K;
  int tiles_m, tiles_n, nk, S, kper;
  int32_t* part;
};

// WM x WN waves over a tile of BM rows of X and BN rows of W.
template <int BM, int BN, int WM, int WN, int NS, bool WHOLE, int TYPE>
__global__ __launch_bounds__(WM* WN* kWaveSize) void i8_gemm_kernel(GemmArgs g) {
  constexpr int kThreads = WM * WN * kWaveSize;
  constexpr int WR = BM / WM, WC = BN / WN;  // of a wave
  constexpr int MI = WR / 32, NJ = WC / 32;
  constexpr int kX = BM * kStepBytes, kW = BN * kStepBytes, kStage = kX + kW;
  constexpr int kPitch = WC * 4 + 16;  // bytes of 32 rows of results in LDS, wave by wave
  // The steps' stages are apart, so that the compiler can tell a copy into one from a read of
  // another.
  __shared__ __attribute__((aligned(1024))) uint8_t s0[kStage], s1[kStage];
  __shared__ __attribute__((aligned(1024))) uint8_t s2[NS > 2 ? kStage : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t s3[NS > 3 ? kStage : 16];
  uint8_t* const st[4] = {s0, s1, s2, s3};
  const int L = xcd_logical_tile(blockIdx.x, gridDim.x);
  const int tiles = g.tiles_m * g.tiles_n;
  const int sp = L / tiles;
  int tm, tn;
  tile_of(L - sp * tiles, g.tiles_m, g.tiles_n, tm, tn);
  const int m0 = tm * BM, n0 = tn * BN;
  const int rows = min(BM, g.M - m0), cols = min(BN, g.N - n0);
  const int kb = sp * g.kper, ke = min(g.nk, kb + g.kper);  // the plan leaves no split empty
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = wave % WM, wn = wave / WM;

  RowCopy<BM, kThreads> cx;
  RowCopy<BN, kThreads> cw;
  constexpr int kCopies = cx.kInstr + cw.kInstr;  // of a wave in a step
  cx.init(g.X + (size_t)m0 * g.K, rows, (uint32_t)g.K, t);
  cw.init(g.W + (size_t)n0 * g.K, cols, (uint32_t)g.K, t);
  // steps past the last copy zeros, without an access of memory, and are not read
  auto issue = [&](uint8_t* stage, int ks) __attribute__((always_inline)) {
    const int k = min(ks, ke - 1);
    const int left = ks < ke ? g.K - k * kStepBytes : 0;
    cx.issue(stage, k, left, wave);
    cw.issue(stage + kX, k, left, wave);
  };

  int16v acc[MI][NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
  struct Operands {
    int4v x[MI], w[NJ];
  };
  const int rx = wm * WR + (lane & 31), rw = wn * WC + (lane & 31);
  // chunk 2 * q + lane / 32 of a row in quarter q; 32 rows on the swizzle is the same
  const int xo = rx * kStepBytes + (((lane >> 5) ^ swz_row(rx)) << 4);
  const int wo = kX + rw * kStepBytes + (((lane >> 5) ^ swz_row(rw)) << 4);
  auto read = [&](Operands& o, const uint8_t* stage, int q) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
      o.x[i] = *reinterpret_cast<const int4v*>(stage + (xo ^ (q << 5)) + 32 * i * kStepBytes);
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      o.w[j] = *reinterpret_cast<const int4v*>(stage + (wo ^ (q << 5)) + 32 * j * kStepBytes);
  };
  auto multiply = [&](const Operands& o) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(o.w[j], o.x[i], acc[i][j], 0, 0, 0);
  };
  // The reads of 32 bytes of a step are issued before the products of the 32 before; a step's
  // last products run over the first reads of the next step and the copies into the stage
  // that this step leaves.
  constexpr int Q = kStepBytes / 32;
  Operands o[WHOLE ? 2 * Q : 2];
  auto step = [&](uint8_t* cur, uint8_t* next, int ks, int half) __attribute__((always_inline)) {
    if constexpr (WHOLE) {
      tile_hand_over<kCopies*(NS - 2)>();
#pragma unroll
      for (int q = 0; q < Q; ++q) read(o[Q * (1 - half) + q], next, q);
      issue(cur, ks + NS);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int q = 0; q < Q; ++q) multiply(o[Q * half + q]);
      __builtin_amdgcn_sched_barrier(0);
    } else {
#pragma unroll
      for (int q = 0; q < Q - 1; ++q) {
        read(o[(q + 1) & 1], cur, q + 1);
        __builtin_amdgcn_sched_barrier(0);
        multiply(o[q & 1]);
        __builtin_amdgcn_sched_barrier(0);
      }
      tile_hand_over<kCopies*(NS - 2)>();
      read(o[0], next, 0);
      issue(cur, ks + NS);
      __builtin_amdgcn_sched_barrier(0);
      multiply(o[1]);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
#pragma unroll
  for (int u = 0; u < NS; ++u) issue(st[u], kb + u);
  tile_hand_over<kCopies*(NS - 1)>();
#pragma unroll
  for (int q = 0; q < (WHOLE ? Q : 1); ++q) read(o[q], s0, q);
  // stages and operand sets alternate at compile time
  constexpr int U = WHOLE && NS % 2 ? 2 * NS : NS;
  int ks = kb;
  for (; ks + U <= ke; ks += U)
#pragma unroll
    for (int u = 0; u < U; ++u) step(st[u % NS], st[(u + 1) % NS], ks + u, u & 1);
#pragma unroll
  for (int u = 0; u < U - 1; ++u)
    if (ks + u < ke) step(st[u % NS], st[(u + 1) % NS], ks + u, u & 1);
  tile_hand_over<0>();  // the last copies have landed before results go where they went

  // A 32 x 32 result has rows of W along its registers: lane l holds row l % 32 of X, register
  // r column 8 * (r / 4) + 4 * (l / 32) + r % 4.
  const int mw = m0 + wm * WR, rlive = rows - wm * WR;
  const int nw = n0 + wn * WC;
  const int lr = lane & 31, l4 = 4 * (lane >> 5);
  if (g.S > 1) {
    int32_t* dst = g.part + (size_t)sp * g.M * g.N;
#pragma unroll
    for (int i = 0; i < MI; ++i)
      if (32 * i + lr < rlive)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int n = nw + 32 * j + 8 * q + l4;
            if (n < g.N)
              *reinterpret_cast<int4v*>(dst + (size_t)(mw + 32 * i + lr) * g.N + n) =
                  int4v{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                        acc[i][j][4 * q + 3]};
          }
    return;
  }
  // Results pass through the wave's own part of LDS, 32 rows at a time, and leave in 16-byte
  // pieces.
  constexpr int kFit = kStage / (32 * kPitch);  // waves whose results fit a stage
  static_assert(kFit * NS >= WM * WN, "results fit the stages");
  uint8_t* out = s0;
#pragma unroll
  for (int u = 1; u < NS; ++u)
    if (wave / kFit == u) out = st[u];
  out += wave % kFit * (32 * kPitch);
  typedef typename Val<TYPE>::T T;
  constexpr int kPer = 16 / sizeof(T);         // values of a piece
  constexpr int kPieces = WC / kPer;           // of a row
  float sw[NJ][4][4];
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        sw[j][q][e] = g.sw[min(nw + 32 * j + 8 * q + l4, g.N - 4) + e];
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const float s = g.sx[min(mw + 32 * i + lr, g.M - 1)];
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        T y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          y[e] = Val<TYPE>::put((float)acc[i][j][4 * q + e] * s * sw[j][q][e]);
        __builtin_memcpy(__builtin_assume_aligned(
                             out + lr * kPitch + (32 * j + 8 * q + l4) * (int)sizeof(T),
                             sizeof(y)),
                         y, sizeof(y));
      }
#pragma unroll
    for (int p0 = 0; p0 < 32 * kPieces; p0 += kWaveSize) {
      const int r = (p0 + lane) / kPieces, pc = (p0 + lane) % kPieces;
      const int n = nw + kPer * pc;
      if (32 * i + r < rlive && n < g.N)
        *reinterpret_cast<uint4*>(static_cast<T*>(g.Y) + (size_t)(mw + 32 * i + r) * g.N + n) =
            *reinterpret_cast<const uint4*>(out + r * kPitch + 16 * pc);
    }
  }
}

template <int BM, int BN, int WM, int WN, int NS, bool WHOLE>
void launch_tile(const GemmArgs& g, int type, hipStream_t st) {
  i8_by_type(type, [&](auto t) {
    hipLaunchKernelGGL((i8_gemm_kernel<BM, BN, WM, WN, NS, WHOLE, decltype(t)::value>),
                       dim3((unsigned)(g.tiles_m * g.tiles_n * g.S)), dim3(WM * WN * kWaveSize), 0,
                       st, g);
  });
}

}  // namespace

// Tiles, measured (us a call on the GPU, bf16 results): 2048 rows of 4096 x 11008: 256 x 192 101 to
// 106, 128 x 256 102 to 103, 128 x 128 121 (on another GPU 95, 104 and 121); of 4096 x 4096: 44,
// 37.4, 44; 777 of 4096 x 4096: 38.5, 27.5, 20.8, and 64 x 128 22.9; of 5120 x 1536: 64 x 128 17.5,
// 128 x 128 in 3 splits 21.9, 64 x 64 19.7; 130 of 4096 x 4096: 64 x 64 9.8, 64 x 128 12.9,
// 128 x 128 in 4 splits 18.2; 33 of 4096 x 11008: 64 x 64 10.4, 32 x 64 12.2, 64 x 128 in 2 splits
// 13.5; 20 of 4096 x 4096: 32 x 64 8.5, 64 x 64 in 4 splits 8.7.
constexpr I8Tile kTiles[] = {{256, 192, 0.90, 0.90, 0.50},
                             {128, 256, 0.70, 0.70, 0.30},
                             {128, 128, 0.46, 0.46, 0.14},
                             {64, 128, 0.35, 0.27, 0.04},
                             {64, 64, 0.20, 0.19, 0.02},
                             {32, 64, 0.13, 0.11, 0.04}};

I8Plan plan_i8_gemm(int M, int N, int K) {
  I8Plan p{};
  p.strip = M <= kI8FewRows;
  if (p.strip) {
    p.S = 1;
    p.kper = (K + 127) / 128;
    return p;
  }
  plan_i8_tiles(p, kTiles, M, N, (K + kStepBytes - 1) / kStepBytes);
  if (p.S > 1) p.ws_bytes = (size_t)p.S * M * N * sizeof(int32_t);
  return p;
}

hipError_t launch_i8_gemm(const int8_t* X, const float* sx, const int8_t* W, const float* sw,
                          void* Y, int type, int M, int N, int K, void* ws, const I8Plan& p,
                          hipStream_t st) {
  if (p.strip) return launch_i8_strip(X, sx, W, sw, Y, type, M, N, K, st);
  const GemmArgs g{X, sx, W, sw, Y, M, N, K, p.tiles_m, p.tiles_n, p.nk, p.S, p.kper,
                   static_cast<int32_t*>(ws)};
  if ((long long)p.tiles_m * p.tiles_n * p.S > 0x3fffffLL) return hipErrorInvalidValue;
  switch (p.tile) {
    case 0: launch_tile<256, 192, 4, 2, 2, false>(g, type, st); break;
    case 1: launch_tile<128, 256, 2, 4, 3, false>(g, type, st); break;
    case 2: launch_tile<128, 128, 2, 4, 4, false>(g, type, st); break;
    case 3: launch_tile<64, 128, 2, 4, 3, true>(g, type, st); break;
    case 4: launch_tile<64, 64, 2, 2, 4, true>(g, type, st); break;
    default: launch_tile<32, 64, 1, 2, 4, true>(g, type, st);
  }
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || p.S == 1) return err;
  return launch_i8_finish(g.part, sx, sw, Y, type, M, N, p.S, st);
}

}  // namespace q4
