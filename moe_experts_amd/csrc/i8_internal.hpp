// Plans and launchers of the 8-bit operators: rows of int8 with one fp32 scale
// each, their products and the gradients of those products.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "q4moe.h"

namespace q4 {

// ---- rows (i8_rows.hip) ------------------------------------------------------
// Which form of a row kernel serves a shape: threads of a workgroup, pieces of eight values that
// a lane holds, passes over the data.
struct I8RowsPlan {
  int threads, pieces, passes;
};
I8RowsPlan plan_i8_quantize(int M, int K);
I8RowsPlan plan_i8_gradient_rows(int ld);
I8RowsPlan plan_i8_gradient_columns(int M, int N, int ld);
hipError_t launch_i8_quantize(const void* X, int type, int8_t* Q, float* scale, int M, int K,
                              hipStream_t st);
hipError_t launch_i8_dequantize(const int8_t* Q, const float* scale, void* X, int type, int M,
                                int K, hipStream_t st);

// ---- few rows (i8_strip.hip) -------------------------------------------------
// Y = X . W^T for X of up to kI8FewRows rows, scaled and rounded.
constexpr int kI8FewRows = 16;
hipError_t launch_i8_strip(const int8_t* X, const float* sx, const int8_t* W, const float* sw,
                           void* Y, int type, int M, int N, int K, hipStream_t st);
struct I8GemvPlan {
  bool fused;      // the rows are quantized by every workgroup, not by a launch of their own
  size_t off_s;    // else: int8 [M][K], then fp32 [M]
  size_t ws_bytes;
};
I8GemvPlan plan_i8_gemv(int M, int N, int K);
hipError_t launch_i8_gemv(const float* x, const int8_t* W, const float* sw, float* y, int M, int N,
                          int K, void* ws, const I8GemvPlan& p, hipStream_t st);

// ---- many rows (i8_gemm.hip, i8_gradient.hip) ---------------------------------
// Result [rows][cols] by tiles of BM x BN, K steps of 128 bytes of the left operand, S splits of
// the contraction (32-bit partial sums [S][rows][cols] in ws).
struct I8Plan {
  bool strip;      // few rows or little work, by a kernel of its own (BM is 0)
  int tile;        // of those compiled
  int BM, BN;
  int tiles_m, tiles_n;
  int nk;          // K steps of the whole contraction
  int S, kper;     // splits, K steps of one
  size_t off_a;    // gradients: the left operand, fp16 [rows][ld]
  size_t off_rs;   // gradients: fp32 [rows], what a row of the product is multiplied by
  size_t off_a2;   // gradients: what that has lost, bf16 [rows][ld], of the rows that have lost any
  size_t off_lost; // gradients: uint32 [rows], the sum of it
  size_t off_max;  // weight gradient: uint32 [2][chunks of M][N]
  size_t off_part;
  int ld;          // gradients: values of a row of the left operand
  size_t ws_bytes;
};

// What a tile costs. A CU that has n of them to do takes n * (each + busy * load) us a K step,
// load being the share of what n on every CU would be (the clock falls as more of the GPU is
// busy), or `alone` with one. They come from sweeps of tiles and splits.
struct I8Tile {
  int BM, BN;
  double alone, each, busy;
};
// The tile and the number of splits by the time a CU with the most work takes: its steps, 3 us
// and 0.8 a tile for the start and the results; splits cost the partial sums, written and read
// at 4.5 TB/s, and a kernel that adds them.
template <int COUNT>
void plan_i8_tiles(I8Plan& p, const I8Tile (&tiles)[COUNT], int rows, int cols, int nk) {
  double best = 1e30;
  p.nk = nk;
  for (int t = 0; t < COUNT; ++t) {
    const int tm = (rows + tiles[t].BM - 1) / tiles[t].BM;
    const int tn = (cols + tiles[t].BN - 1) / tiles[t].BN;
    for (int s = 1; s <= 32 && (s == 1 || nk / s >= 2); ++s) {
      const int kper = (nk + s - 1) / s;
      if ((nk + kper - 1) / kper != s) continue;
      const double count = (double)tm * tn * s;
      if (s > 1 && count > 4096) continue;
      const double n = (double)(((long long)count + 255) / 256);
      const double load = count / (256.0 * n);
      const double step =
          n == 1 ? tiles[t].alone + tiles[t].busy * load : n * (tiles[t].each + tiles[t].busy * load);
      double cost = kper * step + 3.0 + 0.8 * n;
      if (s > 1) cost += 4.0 + s * (double)rows * cols * 8.0 / 4.5e6;
      if (cost < best) {
        best = cost;
        p.tile = t;
        p.BM = tiles[t].BM;
        p.BN = tiles[t].BN;
        p.tiles_m = tm;
        p.tiles_n = tn;
        p.S = s;
        p.kper = kper;
      }
    }
  }
}

I8Plan plan_i8_gemm(int M, int N, int K);
hipError_t launch_i8_gemm(const int8_t* X, const float* sx, const int8_t* W, const float* sw,
                          void* Y, int type, int M, int N, int K, void* ws, const I8Plan& p,
                          hipStream_t st);

I8Plan plan_i8_backward(int M, int N, int K);
// the row kernel in front of the tiles; zeros where there is none
I8RowsPlan plan_i8_backward_rows(int M, int N, int K);
hipError_t launch_i8_backward(const uint16_t* dY, const int8_t* W, const float* sw, uint16_t* dX,
                              int M, int N, int K, void* ws, const I8Plan& p, hipStream_t st);

I8Plan plan_i8_backward_weight(int M, int N, int K);
I8RowsPlan plan_i8_backward_weight_rows(int M, int N, int K);
hipError_t launch_i8_backward_weight(const uint16_t* dY, const int8_t* X, const float* sx,
                                     uint16_t* dW, int M, int N, int K, void* ws, const I8Plan& p,
                                     hipStream_t st);

// ---- gradients of few rows or little work (i8_few_gradient.hip) -------------------
// Plans a gradient of rows x cols over `depth`, in at most `splits`; false: by tiles.
constexpr int kFewSplits = 64;
bool plan_i8_few_gradient(I8Plan& p, int rows, int cols, int depth, int splits);
// dY [depth][rows] (transposed) or [rows][depth], scale [depth], B [depth][cols]
hipError_t launch_i8_few_gradient(const uint16_t* dY, bool transposed, const float* scale,
                                  const int8_t* B, uint16_t* out, int rows, int cols, int depth,
                                  float* part, const I8Plan& p, hipStream_t st);

// ---- left operands of the gradients, sums of splits (i8_rows.hip) --------------
struct LeftOperand {
  uint16_t* a;     // fp16 [rows][ld]
  uint16_t* a2;    // what its values below fp16's normal range lost (i8_lost.hpp), bf16 [rows][ld],
                   // where lost[row] is not 0
  float* rs;       // [rows]
  uint32_t* lost;  // [rows]
  int ld;
};
// a[m][n] = fp16(dY[m][n] * sw[n] * 2^e), n < ld (zero past N), rs[m] = 2^-e
hipError_t launch_i8_gradient_rows(const uint16_t* dY, const float* sw, const LeftOperand& l, int M,
                                   int N, hipStream_t st);
// a[n][m] = fp16(dY[m][n] * sx[m] * 2^e), m < ld (zero past M), rs[n] = 2^-e; scratch: the largest
// and the least magnitudes of a column in each of i8_max_chunks(M, N) chunks of the rows
int i8_max_chunks(int M, int N);
hipError_t launch_i8_gradient_columns(const uint16_t* dY, const float* sx, const LeftOperand& l,
                                      uint32_t* scratch, int M, int N, hipStream_t st);
hipError_t launch_i8_finish(const int32_t* part, const float* sx, const float* sw, void* Y,
                            int type, int M, int N, int S, hipStream_t st);
// rs may be null: sums as they are
hipError_t launch_i8_gradient_finish(const float* part, const float* rs, uint16_t* out, int rows,
                                     int cols, int S, hipStream_t st);

}  // namespace q4
