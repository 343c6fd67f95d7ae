// Plans and launchers of the dense feed-forward operators over frozen Q4_0
// weights: the gated block, the projection with adapters and the gradients.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "q4_internal.hpp"

namespace q4 {

// ---- adapters --------------------------------------------------------------
struct Adapters {
  const uint16_t* A;    // fp16 [L][R][K]
  const uint16_t* B;    // fp16 [L][N][R]
  const int32_t* ids;   // [M], outside [0, L): no adapter
  const float* scale;   // [L]
  int R, L;
};

// ---- few rows (ffn_strip.hip) ------------------------------------------------
// Split-K partial sums part[mats][S][M][N] of X . W0 and, with W1, X . W1, for
// fp32 X of up to 8 rows or fp16 X of up to 64 (K a multiple of 32). With ad, the
// same launch forms the adapters' narrow product t[M][R] (scale included).
struct StripPlan {
  int DW, strips, steps;
  int base, more;  // splits of a strip: base, the first `more` strips one more
  int S;           // sums, splits of the most
  size_t part_bytes;
};
StripPlan plan_strip(int M, int N, int K, int mats, bool f32);
hipError_t launch_strip(const void* X, const uint8_t* W0, const uint8_t* W1, float* part, int M,
                        int N, int K, bool f32, const StripPlan& p, hipStream_t st,
                        const Adapters* ad = nullptr, float* t = nullptr);

// ---- decode (fp32, M <= 8; ffn_decode.hip) ----------------------------------
// Split-K partial sums part[mats][S][M][N] by the strips or by the GEMV tiles.
struct DecodePlan {
  bool strip;
  StripPlan sp;
  GemvPlan gemv;
  int S;
  size_t off_t;     // adapters: fp32 [M][R] behind the partial sums
  size_t ws_bytes;
};
DecodePlan plan_glu(int M, int N, int K);
hipError_t launch_glu(const float* x, const uint8_t* Wg, const uint8_t* Wu, float* h, int M, int N,
                      int K, int act, void* ws, const DecodePlan& p, hipStream_t st);

DecodePlan plan_gemv_lora(int M, int N, int K, int R);
hipError_t launch_gemv_lora(const float* x, const uint8_t* B, const Adapters& ad, float* y, int M,
                            int N, int K, void* ws, const DecodePlan& p, hipStream_t st);

// ---- prompt and gradient GEMMs (fp16 matrix cores) --------------------------
// C[M][ncols] (one or two matrices) by tiles of BM x 128, K steps of 64, S
// splits of the contraction.
struct FfnPlan {
  bool strip;       // few rows: by the strips (sp), whose partial sums S counts
  StripPlan sp;
  int BM;           // tile rows
  int tiles_m, tiles_n;
  int nk;           // K steps of the whole contraction
  int S, kper;      // splits, K steps of one
  size_t off_part;  // fp32 [mats][S][M][ncols], only when S > 1
  size_t off_tp;    // adapters: fp32 [shares of K][M][R], many rows only
  size_t off_t;     // adapters: fp32 [M][R]
  size_t off_t16;   // adapters: fp16 [M][R], rows scaled to their largest value
  size_t off_ts;    // adapters: fp32 [M], what a row of t16 is multiplied by
  size_t off_a;     // gradients: fp16 [M][mats * N], rows scaled by a power of two
  size_t off_rs;    // gradients: fp32 [M], what a row of the product is multiplied by
  size_t ws_bytes;
};

FfnPlan plan_glu_gemm(int M, int N, int K);
hipError_t launch_glu_gemm(const uint16_t* X, const uint8_t* Wg, const uint8_t* Wu, uint16_t* H,
                           uint16_t* G, uint16_t* U, int M, int N, int K, int act, void* ws,
                           const FfnPlan& p, hipStream_t st);

FfnPlan plan_gemm_lora(int M, int N, int K, int R);
hipError_t launch_gemm_lora(const uint16_t* X, const uint8_t* B, const Adapters& ad, uint16_t* Y,
                            int M, int N, int K, void* ws, const FfnPlan& p, hipStream_t st);

// mats = 2: the gated block (dH, G, U); mats = 1: one projection (dH is dY).
FfnPlan plan_gradient(int M, int N, int K, int mats);
hipError_t launch_gradient(const uint16_t* dH, const uint16_t* G, const uint16_t* U,
                           const uint8_t* W0, const uint8_t* W1, uint16_t* dX, int M, int N, int K,
                           int act, int mats, void* ws, const FfnPlan& p, hipStream_t st);

// ---- row kernels shared by the paths (ffn_rows.hip) -------------------------
// h = act(g) * u from the partial sums part[2][S][M][N] (mn = M * N, N % 32 == 0).
hipError_t launch_glu_finish(const float* part, float* h, size_t mn, int S, int act,
                             hipStream_t st);
hipError_t launch_glu_finish_f16(const float* part, uint16_t* H, uint16_t* G, uint16_t* U,
                                 size_t mn, int S, int act, hipStream_t st);
// t[m][r] = scale[id] * sum_k x[m][k] * A[id][r][k], 0 for a row without adapter,
// or, with t16, t16 and ts (FfnPlan); tp[shares][M][R] is scratch.
int shrink_shares(int M, int K);
hipError_t launch_lora_shrink(const uint16_t* X, const Adapters& ad, float* tp, float* t,
                              uint16_t* t16, float* ts, int M, int K, hipStream_t st);
// y[m][n] = sum_s part[s][m][n] + sum_r t[m][r] * B[id][n][r]
hipError_t launch_lora_finish(const float* part, const float* t, const Adapters& ad, float* y,
                              int M, int N, int S, hipStream_t st);
hipError_t launch_lora_finish_f16(const float* part, const float* t, const Adapters& ad,
                                  uint16_t* Y, int M, int N, int S, hipStream_t st);
// The gradient GEMM's left operand (fp16, rows scaled by a power of two, the
// eight values of a group in the order 0 4 1 5 2 6 3 7) and 1 / scale per row.
hipError_t launch_gradient_rows(const uint16_t* dH, const uint16_t* G, const uint16_t* U,
                                uint16_t* a, float* rs, int M, int N, int act, int mats,
                                hipStream_t st);
hipError_t launch_gradient_finish(const float* part, const float* rs, uint16_t* dX, int M, int K,
                                  int S, hipStream_t st);

}  // namespace q4
