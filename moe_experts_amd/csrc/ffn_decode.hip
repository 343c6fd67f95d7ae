// Decode (fp32, up to 8 rows) of the dense feed-forward operators. The products
// with the Q4_0 matrices leave split-K partial sums; what the operators add is
// in the kernel that sums them.
//   gated block  one launch over both matrices, then h = act(g) * u
//   adapters     the product and t = x . A_id^T in one launch, then y = sum + t . B_id^T
#include "ffn_internal.hpp"

namespace q4 {
namespace {

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

// One and two rows of the gated block go through the GEMV's vector tiles, all
// else through the strips on the matrix cores. Both sides measured: 5120 x 1536
// (two matrices) at 1 row 5.6 us by the tiles, 9.4 by the strips; 4096 x 11008
// (two matrices) at 8 rows 26 us by the GEMV's fp32 matrix-core tiles, 19.5 by
// the strips. With adapters the strips' launch takes the narrow product along:
// 4096 x 4096 at 1 row, rank 16: 9.4 us in one launch, by the tiles 3.1 + 5.6 us
// in two, and a launch more costs the host 2.5 us.
DecodePlan plan_glu(int M, int N, int K) {
  DecodePlan p{};
  p.strip = M >= 3;
  if (p.strip) {
    p.sp = plan_strip(M, N, K, 2, true);
    p.S = p.sp.S;
  } else {
    p.gemv = plan_gemv_pair(M, N, K);
    p.S = p.gemv.S;
  }
  p.ws_bytes = (size_t)2 * p.S * M * N * sizeof(float);
  return p;
}

hipError_t launch_glu(const float* x, const uint8_t* Wg, const uint8_t* Wu, float* h, int M, int N,
                      int K, int act, void* ws, const DecodePlan& p, hipStream_t st) {
  float* part = static_cast<float*>(ws);
  const hipError_t err = p.strip
                             ? launch_strip(x, Wg, Wu, part, M, N, K, true, p.sp, st)
                             : launch_gemv_pair(x, Wg, Wu, M, N, K, part, p.gemv, st);
  if (err != hipSuccess) return err;
  return launch_glu_finish(part, h, (size_t)M * N, p.S, act, st);
}

DecodePlan plan_gemv_lora(int M, int N, int K, int R) {
  DecodePlan p{};
  p.strip = true;
  p.sp = plan_strip(M, N, K, 1, true);
  p.S = p.sp.S;
  p.off_t = align256(p.sp.part_bytes);
  p.ws_bytes = p.off_t + (size_t)M * R * sizeof(float);
  return p;
}

hipError_t launch_gemv_lora(const float* x, const uint8_t* B, const Adapters& ad, float* y, int M,
                            int N, int K, void* ws, const DecodePlan& p, hipStream_t st) {
  float* part = static_cast<float*>(ws);
  float* t = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + p.off_t);
  const hipError_t err = launch_strip(x, B, nullptr, part, M, N, K, true, p.sp, st, &ad, t);
  if (err != hipSuccess) return err;
  return launch_lora_finish(part, t, ad, y, M, N, p.S, st);
}

}  // namespace q4
