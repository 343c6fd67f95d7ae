// Decode (fp32, up to 8 rows) of the dense feed-forward operators. The products
// with the Q4_0 matrices leave split-K partial sums; what the operators add is
// in the kernel that sums them.
//   gated block  one launch over both matrices, then h = act(g) * u
//   adapters     t = x . A_id^T, the product, then y = sum + t . B_id^T
#include "ffn_internal.hpp"

namespace q4 {
namespace {

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

// One and two rows go through the GEMV's vector tiles, more through the strips
// on the matrix cores. Both sides measured: 5120 x 1536 (two matrices) at 1 row
// 5.6 us by the tiles, 9.4 by the strips; 4096 x 11008 (two matrices) at 8 rows
// 26 us by the GEMV's fp32 matrix-core tiles, 19.5 by the strips.
DecodePlan plan_decode(int M, int N, int K, int mats) {
  DecodePlan p{};
  p.strip = M >= 3;
  if (p.strip) {
    p.sp = plan_strip(M, N, K, mats, true);
    p.S = p.sp.S;
  } else {
    p.gemv = plan_gemv_part(M, N, K, mats);
    p.S = p.gemv.S;
  }
  p.off_t = align256((size_t)mats * p.S * M * N * sizeof(float));
  p.ws_bytes = p.off_t;
  return p;
}

hipError_t launch_products(const float* x, const uint8_t* W0, const uint8_t* W1, float* part,
                           int M, int N, int K, const DecodePlan& p, hipStream_t st) {
  if (p.strip) return launch_strip(x, W0, W1, part, M, N, K, true, p.sp, st);
  return launch_gemv_part(x, W0, W1, M, N, K, part, p.gemv, st);
}

}  // namespace

DecodePlan plan_glu(int M, int N, int K) { return plan_decode(M, N, K, 2); }

hipError_t launch_glu(const float* x, const uint8_t* Wg, const uint8_t* Wu, float* h, int M, int N,
                      int K, int act, void* ws, const DecodePlan& p, hipStream_t st) {
  float* part = static_cast<float*>(ws);
  const hipError_t err = launch_products(x, Wg, Wu, part, M, N, K, p, st);
  if (err != hipSuccess) return err;
  return launch_glu_finish(part, h, (size_t)M * N, p.S, act, st);
}

DecodePlan plan_gemv_lora(int M, int N, int K, int R) {
  DecodePlan p = plan_decode(M, N, K, 1);
  p.ws_bytes = p.off_t + (size_t)M * R * sizeof(float);
  return p;
}

hipError_t launch_gemv_lora(const float* x, const uint8_t* B, const Adapters& ad, float* y, int M,
                            int N, int K, void* ws, const DecodePlan& p, hipStream_t st) {
  float* part = static_cast<float*>(ws);
  float* t = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + p.off_t);
  hipError_t err = launch_lora_shrink(x, ad, t, M, K, st);
  if (err != hipSuccess) return err;
  err = launch_products(x, B, nullptr, part, M, N, K, p, st);
  if (err != hipSuccess) return err;
  return launch_lora_finish(part, t, ad, y, M, N, p.S, st);
}

}  // namespace q4
