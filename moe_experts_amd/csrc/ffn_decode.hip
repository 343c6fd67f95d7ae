// Decode (fp32, up to 8 rows) of the dense feed-forward operators: the GEMV
// tiles of gemv_vector.hpp and gemv_mfma_q4_0.hip do the products with the
// Q4_0 matrices and leave split-K partial sums; what the operators add is in
// the kernel that sums them.
//   gated block  one launch over both matrices, then h = act(g) * u
//   adapters     t = x . A_id^T, the GEMV, then y = sum + t . B_id^T
#include "ffn_internal.hpp"

namespace q4 {

GemvPlan plan_glu(int M, int N, int K) { return plan_gemv_pair(M, N, K); }

hipError_t launch_glu(const float* x, const uint8_t* Wg, const uint8_t* Wu, float* h, int M, int N,
                      int K, int act, void* ws, const GemvPlan& p, hipStream_t st) {
  const hipError_t err = launch_gemv_pair(x, Wg, Wu, M, N, K, ws, p, st);
  if (err != hipSuccess) return err;
  return launch_glu_finish(static_cast<const float*>(ws), h, (size_t)M * N, p.S, act, st);
}

GemvLoraPlan plan_gemv_lora(int M, int N, int K, int R) {
  GemvLoraPlan p;
  p.gemv = plan_gemv(M, N, K);
  p.off_t = ((size_t)p.gemv.S * M * N * sizeof(float) + 255) / 256 * 256;
  p.ws_bytes = p.off_t + (size_t)M * R * sizeof(float);
  return p;
}

hipError_t launch_gemv_lora(const float* x, const uint8_t* B, const Adapters& ad, float* y, int M,
                            int N, int K, void* ws, const GemvLoraPlan& p, hipStream_t st) {
  float* part = static_cast<float*>(ws);
  float* t = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + p.off_t);
  hipError_t err = launch_lora_shrink(x, ad, t, M, K, st);
  if (err != hipSuccess) return err;
  // with one split the GEMV writes its y argument: the slab
  err = launch_gemv(x, B, part, M, N, K, part, p.gemv, st, false);
  if (err != hipSuccess) return err;
  return launch_lora_finish(part, t, ad, y, M, N, p.gemv.S, st);
}

}  // namespace q4
