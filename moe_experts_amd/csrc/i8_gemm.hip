// 8-bit product of many rows: Y = (X . W^T) * sx * sw, X int8 [M][K], W int8 [N][K], on the
// integer matrix cores (v_mfma_i32_32x32x32_i8). The sums are whole numbers and exact, so
// splits of the contraction change nothing.
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
template <int BM, int BN, int WM, int WN, int TYPE>
__global__ __launch_bounds__(WM* WN* kWaveSize) void i8_gemm_kernel(GemmArgs g) {
  constexpr int kThreads = WM * WN * kWaveSize;
  constexpr int WR = BM / WM, WC = BN / WN;  // of a wave
  constexpr int MI = WR / 32, NJ = WC / 32;
  constexpr int kX = BM * kStepBytes, kW = BN * kStepBytes;
  constexpr int kPitch = WC * 4 + 16;  // bytes of 32 rows of results in LDS, wave by wave
  static_assert(WM * WN * 32 * kPitch <= 2 * (kX + kW), "results fit the stages");
  // Two steps, apart, so that the compiler can tell a copy into one from a read of the other.
  __shared__ __attribute__((aligned(1024))) uint8_t s0[kX + kW];
  __shared__ __attribute__((aligned(1024))) uint8_t s1[kX + kW];
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
  cx.init(g.X + (size_t)m0 * g.K, rows, (uint32_t)g.K, t);
  cw.init(g.W + (size_t)n0 * g.K, cols, (uint32_t)g.K, t);
  // steps past the last repeat it, into a stage that is not read
  auto issue = [&](uint8_t* stage, int ks) __attribute__((always_inline)) {
    const int k = min(ks, ke - 1);
    const int left = g.K - k * kStepBytes;
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
  // The reads of a quarter are issued before the products of the one before; a step's last
  // products run over the first reads of the next step and the copies of the one after.
  Operands o[2];
  auto step = [&](uint8_t* cur, uint8_t* next, int ks) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      read(o[(q + 1) & 1], cur, q + 1);
      __builtin_amdgcn_sched_barrier(0);
      multiply(o[q & 1]);
      __builtin_amdgcn_sched_barrier(0);
    }
    tile_hand_over();
    read(o[0], next, 0);
    issue(cur, ks + 2);
    __builtin_amdgcn_sched_barrier(0);
    multiply(o[1]);
    __builtin_amdgcn_sched_barrier(0);
  };
  issue(s0, kb);
  issue(s1, kb + 1);
  tile_hand_over();
  read(o[0], s0, 0);
  int ks = kb;
  for (; ks + 2 <= ke; ks += 2) {
    step(s0, s1, ks);
    step(s1, s0, ks + 1);
  }
  if (ks < ke) step(s0, s1, ks);
  tile_hand_over();  // the last copies have landed before results go where they went

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
  static_assert(WM * WN / 2 * 32 * kPitch <= kX + kW, "half of the waves in either stage");
  uint8_t* out = (wave & 1 ? s1 : s0) + (wave >> 1) * (32 * kPitch);
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

template <int BM, int BN, int WM, int WN>
void launch_tile(const GemmArgs& g, int type, hipStream_t st) {
  i8_by_type(type, [&](auto t) {
    hipLaunchKernelGGL((i8_gemm_kernel<BM, BN, WM, WN, decltype(t)::value>),
                       dim3((unsigned)(g.tiles_m * g.tiles_n * g.S)), dim3(WM * WN * kWaveSize), 0,
                       st, g);
  });
}

}  // namespace

I8Plan plan_i8_gemm(int M, int N, int K) {
  I8Plan p{};
  p.strip = M <= kI8FewRows;
  if (p.strip) return p;
  p.nk = (K + kStepBytes - 1) / kStepBytes;
  p.BM = p.BN = 128;
  if (M > 1024 && N >= 4096) p.BM = p.BN = 256;
  p.tiles_m = (M + p.BM - 1) / p.BM;
  p.tiles_n = (N + p.BN - 1) / p.BN;
  int s = 1;
  while (p.tiles_m * p.tiles_n * s * 2 <= 320 && p.nk / (2 * s) >= 4) s *= 2;
  p.kper = (p.nk + s - 1) / s;
  p.S = (p.nk + p.kper - 1) / p.kper;
  if (p.S > 1) p.ws_bytes = (size_t)p.S * M * N * sizeof(int32_t);
  return p;
}

hipError_t launch_i8_gemm(const int8_t* X, const float* sx, const int8_t* W, const float* sw,
                          void* Y, int type, int M, int N, int K, void* ws, const I8Plan& p,
                          hipStream_t st) {
  if (p.strip) return launch_i8_strip(X, sx, W, sw, Y, type, M, N, K, st);
  GemmArgs g{X, sx, W, sw, Y, M, N, K, p.tiles_m, p.tiles_n, p.nk, p.S, p.kper,
             static_cast<int32_t*>(ws)};
  if ((long long)p.tiles_m * p.tiles_n * p.S > 0x3fffffLL) return hipErrorInvalidValue;
  if (p.BM == 256)
    launch_tile<256, 256, 2, 4>(g, type, st);
  else
    launch_tile<128, 128, 2, 2>(g, type, st);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || p.S == 1) return err;
  return launch_i8_finish(g.part, sx, sw, Y, type, M, N, p.S, st);
}

}  // namespace q4
