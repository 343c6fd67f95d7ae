// 8-bit product of few rows: Y = (X . W^T) * sx * sw for up to 16 rows of X, and the
// decode form that takes fp32 rows and quantizes them itself.
//
// A workgroup owns 16 rows of W (columns of Y) and its four waves share out the
// contraction. v_mfma_i32_16x16x64_i8 takes 16 bytes of one row in a lane for both operands,
// so the weights go from memory straight into its registers, 64 bytes of each of 16 rows a
// load, and nothing but the sums passes through LDS: they are whole numbers, so the order in
// which the waves' are added does not matter.
//
// Bound by the weights' way from memory, 16 MB in FIG1 us and 45 MB in FIG2
#include <algorithm>

#include "i8_device.hpp"
#include "i8_internal.hpp"

namespace q4 {
namespace {

constexpr int kWaves = 4;
constexpr int kStripThreads = kWaves * kWaveSize;
constexpr uint32_t kOut = 0x80000000u;  // past the end of any array
constexpr int kFusedValues = 16384;     // of x, in the LDS of a workgroup that quantizes them
constexpr int kFusedPieces = kFusedValues / 8 / kStripThreads;

struct StripArgs {
  const int8_t* X;   // or, fused, fp32 x
  const float* xf;
  const float* sx;
  const int8_t* W;
  const float* sw;
  void* Y;
  int M, N, K;
  int blocks;
};

// Fused: all of x in registers, the largest of each row by LDS, int8 into xq, rows `pitch`
// bytes apart.
struct FusedRows {
  float x[kFusedPieces][8];
  __device__ __forceinline__ void load(const StripArgs& g) {
    const int total = g.M * g.K / 8;
#pragma unroll
    for (int i = 0; i < kFusedPieces; ++i) {
      const int p = i * kStripThreads + (int)threadIdx.x;
      if (p < total) __builtin_memcpy(x[i], g.xf + (size_t)p * 8, 32);
    }
  }
  __device__ __forceinline__ void quantize(const StripArgs& g, uint8_t* __restrict__ xq, int pitch,
                                           uint32_t* __restrict__ big, float* __restrict__ sx) {
    const int t = threadIdx.x;
    const int total = g.M * g.K / 8;
    if (t < Q4_GEMV_MAX_M) big[t] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kFusedPieces; ++i) {
      const int p = i * kStripThreads + t;
      if (p - (t & 63) >= total) break;  // the whole wave
      const int row = min(p, total - 1) * 8 / g.K;
      uint32_t b = 0;
      if (p < total)
#pragma unroll
        for (int e = 0; e < 8; ++e) b = max(b, magnitude(x[i][e]));
      const int row0 = __builtin_amdgcn_readfirstlane(row);
      if (__all(row == row0)) {
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) b = max(b, (uint32_t)__shfl_xor((int)b, o));
        if ((t & 63) == 0) atomicMax(&big[row0], b);
      } else {
        atomicMax(&big[row], b);
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kFusedPieces; ++i) {
      const int p = i * kStripThreads + t;
      if (p < total) {
        const int row = p * 8 / g.K;
        const RowScale rs = row_scale(big[row]);
        uint32_t q[2];
        to_int8<8>(x[i], rs, q);
        *reinterpret_cast<uint2*>(xq + row * pitch + (p * 8 - row * g.K)) = make_uint2(q[0], q[1]);
        if (p * 8 == row * g.K) sx[row] = rs.s;
      }
    }
    __syncthreads();
  }
};

template <int TYPE, bool FUSED>
__global__ __launch_bounds__(kStripThreads) void i8_few_rows_kernel(StripArgs g) {
  constexpr int U = 4;  // loads of a piece; two pieces are in flight
  // rows of K rounded up to 64, and 16 bytes more; K % 16 == 0 and M * K <= kFusedValues
  constexpr int kXq = FUSED ? kFusedValues + Q4_GEMV_MAX_M * (64 + 16) : 16;
  __shared__ __attribute__((aligned(16))) uint8_t xq[kXq];
  __shared__ uint32_t big[Q4_GEMV_MAX_M];
  __shared__ float sxq[Q4_GEMV_MAX_M];
  __shared__ __attribute__((aligned(16))) int4v sums[kWaves][kWaveSize];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int block = (int)(blockIdx.y * gridDim.x + blockIdx.x);
  if (block >= g.blocks) return;  // the whole workgroup, before any barrier
  const int n0 = block * 16;
  const int K = g.K;
  const int nk = (K + 63) / 64, per = (nk + kWaves - 1) / kWaves;
  const int kb = min(nk, wave * per), ke = min(nk, kb + per);
  const __amdgpu_buffer_rsrc_t rw =
      make_rsrc(g.W + (size_t)n0 * K, (uint32_t)min(16, g.N - n0) * (uint32_t)K);
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(g.X, FUSED ? 0u : (uint32_t)g.M * (uint32_t)K);
  const int kl = 16 * (lane >> 4);
  const uint32_t row = (uint32_t)(lane & 15) * (uint32_t)K + (uint32_t)kl;
  const int pitch = nk * 64 + 16;

  // x first: loads return in order, and the weights are many
  FusedRows rows;
  if constexpr (FUSED) rows.load(g);
  struct Piece {
    int4v w[U], x[FUSED ? 1 : U];
  };
  auto load = [&](Piece& p, int s0) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int s = s0 + u;
      // steps of another wave, values past the row and rows past the last read zeros
      const uint32_t o = s < ke && s * 64 + kl < K ? row : kOut;
      const uint32_t so = (uint32_t)min(s, nk - 1) * 64u;
      if constexpr (!FUSED)
        p.x[u] =
            __builtin_bit_cast(int4v, __builtin_amdgcn_raw_buffer_load_b128(rx, o, so, 0));
      p.w[u] = __builtin_bit_cast(int4v, __builtin_amdgcn_raw_buffer_load_b128(rw, o, so, 0));
    }
  };
  int4v acc = int4v{0, 0, 0, 0};
  const int token = FUSED ? min(lane & 15, g.M - 1) : 0;  // rows past the last are not kept
  auto multiply = [&](const Piece& p, int s0) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      int4v x;
      if constexpr (FUSED)
        x = *reinterpret_cast<const int4v*>(xq + token * pitch + min(s0 + u, nk - 1) * 64 + kl);
      else
        x = p.x[u];
      acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(p.w[u], x, acc, 0, 0, 0);
    }
  };
  Piece p[2];
  load(p[0], kb);
  load(p[1], kb + U);
  if constexpr (FUSED) rows.quantize(g, xq, pitch, big, sxq);
  for (int s = kb; s < ke; s += 2 * U) {
    multiply(p[0], s);
    load(p[0], s + 2 * U);
    multiply(p[1], s + U);
    load(p[1], s + 3 * U);
  }
  sums[wave][lane] = acc;
  __syncthreads();
  // lane l of a 16 x 16 result holds row l % 16 of X and four neighbouring columns
  const int m = lane & 15, n = n0 + 4 * (lane >> 4);
  if (wave != 0 || m >= g.M || n >= g.N) return;
  int4v v = sums[0][lane];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) v += sums[w][lane];
  const float s = FUSED ? sxq[m] : g.sx[m];
  typename Val<TYPE>::T y[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = Val<TYPE>::put((float)v[e] * s * g.sw[n + e]);
  typename Val<TYPE>::T* dst = static_cast<typename Val<TYPE>::T*>(g.Y) + (size_t)m * g.N + n;
  __builtin_memcpy(__builtin_assume_aligned(dst, sizeof(y)), y, sizeof(y));
}

template <int TYPE, bool FUSED>
hipError_t launch(StripArgs g, hipStream_t st) {
  g.blocks = (g.N + 15) / 16;
  // two dimensions: one of the widest matrices' workgroups would pass 2^32 lanes
  const int x = std::min(g.blocks, 1 << 20);
  hipLaunchKernelGGL((i8_few_rows_kernel<TYPE, FUSED>), dim3(x, (g.blocks + x - 1) / x),
                     dim3(kStripThreads), 0, st, g);
  return hipGetLastError();
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

hipError_t launch_i8_strip(const int8_t* X, const float* sx, const int8_t* W, const float* sw,
                           void* Y, int type, int M, int N, int K, hipStream_t st) {
  const StripArgs g{X, nullptr, sx, W, sw, Y, M, N, K, 0};
  hipError_t err = hipSuccess;
  i8_by_type(type, [&](auto t) { err = launch<decltype(t)::value, false>(g, st); });
  return err;
}

I8GemvPlan plan_i8_gemv(int M, int, int K) {
  I8GemvPlan p{};
  p.fused = (long long)M * K <= kFusedValues;
  if (!p.fused) {
    p.off_s = align256((size_t)M * K);
    p.ws_bytes = p.off_s + (size_t)M * sizeof(float);
  }
  return p;
}

hipError_t launch_i8_gemv(const float* x, const int8_t* W, const float* sw, float* y, int M, int N,
                          int K, void* ws, const I8GemvPlan& p, hipStream_t st) {
  if (p.fused) {
    const StripArgs g{nullptr, x, nullptr, W, sw, y, M, N, K, 0};
    return launch<Q4_TYPE_F32, true>(g, st);
  }
  int8_t* q = static_cast<int8_t*>(ws);
  float* s = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + p.off_s);
  const hipError_t err = launch_i8_quantize(x, Q4_TYPE_F32, q, s, M, K, st);
  if (err != hipSuccess) return err;
  return launch_i8_strip(q, s, W, sw, y, Q4_TYPE_F32, M, N, K, st);
}

}  // namespace q4
