// 8-bit product of few rows: Y = (X . W^T) * sx * sw for up to 16 rows of X, and the
// decode form that takes fp32 rows and quantizes them itself.
//
// A workgroup owns 16 rows of W (columns of Y) and its four waves share out the contraction.
// A wave copies 128 bytes of each of the 16 rows a step, memory -> LDS, several steps ahead,
// into a part of LDS of its own: nothing is waited for but its own copies. It multiplies them
// by v_mfma_i32_16x16x64_i8. The waves' sums meet in LDS; they are whole numbers, so their
// order does not matter.
//
// Bound by the weights' way from memory. With the weights loaded straight into the matrix
// instruction's registers (16 rows of 64 bytes a load): 8 rows of 11008 x 4096 12.1 us, by
// copies (8 rows of 128 bytes each) 9.2 to 9.7, 4.7 to 4.9 TB/s; a row of 4096 x 4096 4.9 and 4.6
// to 4.9.
//
// Stages: 48 KiB of them, so that three workgroups fit a CU: four steps of up to 8 rows, three of
// 16. A fourth step of 16 rows leaves two workgroups (4096 x 11008 9.55 -> 10.5 us; 11008 x 4096
// the same, 10.4), a third of 8 does no better (11008 x 4096 9.7 both, one row 9.3 and 9.2), two
// do worse (10.3, 10.7 of 16 rows). With the quantized rows in LDS two to four steps are the same
// (a row of 4096 x 4096 6.1 to 6.2, of 8192 x 4096 10.3 to 10.6).
//
// fp32 rows of up to kFusedValues values in all are quantized by every workgroup for itself
// while its first weights are on their way: a row of 4096 for 4096 x 4096 6.2 to 6.5 us, against
// 4.7 and 3.2 for a launch that quantizes and the time between the two. With more values it
// takes longer than that launch (4 rows of 4096: 11.0 against 8.9).
#include "i8_device.hpp"
#include "i8_internal.hpp"
#include "i8_tile.hpp"

namespace q4 {
namespace {

constexpr int kWaves = 4;
constexpr int kStripThreads = kWaves * kWaveSize;
constexpr int kFusedValues = 8192;  // of x, where every workgroup quantizes them for itself
constexpr int kFusedPieces = kFusedValues / 8 / kStripThreads;

struct StripArgs {
  const int8_t* X;   // or, fused, fp32 x
  const float* xf;
  const float* sx;
  const int8_t* W;
  const float* sw;
  void* Y;
  int M, N, K;
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
    lds_only_barrier();
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
    lds_only_barrier();
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
    lds_only_barrier();
  }
};

// XROWS: rows of X that a wave copies, 8 or 16; 0 for the fused form.
template <int TYPE, int XROWS, int NS>
__global__ __launch_bounds__(kStripThreads) void i8_few_rows_kernel(StripArgs g) {
  constexpr bool FUSED = XROWS == 0;
  constexpr int kCopies = 2 + XROWS / 8;           // of a step, eight rows each
  constexpr int kStage = kCopies * 1024;           // of a wave
  // rows of K rounded up to 128, and 16 bytes more; K % 16 == 0 and M * K <= kFusedValues
  constexpr int kXq = FUSED ? kFusedValues + Q4_GEMV_MAX_M * (128 + 16) : 16;
  __shared__ __attribute__((aligned(16))) uint8_t xq[kXq];
  __shared__ uint32_t big[Q4_GEMV_MAX_M];
  __shared__ float sxq[Q4_GEMV_MAX_M];
  __shared__ __attribute__((aligned(16))) int4v sums[kWaves][kWaveSize];
  // The steps' stages are apart, so that the compiler can tell a copy into one from a read of
  // another; in each every wave has its own part.
  __shared__ __attribute__((aligned(1024))) uint8_t s0[kWaves * kStage], s1[kWaves * kStage];
  __shared__ __attribute__((aligned(1024))) uint8_t s2[NS > 2 ? kWaves * kStage : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t s3[NS > 3 ? kWaves * kStage : 16];
  uint8_t* const st[4] = {s0, s1, s2, s3};
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = (int)blockIdx.x * 16;
  const int K = g.K;
  const int nk = (K + 127) / 128, per = (nk + kWaves - 1) / kWaves;
  const int kb = min(nk, wave * per), ke = min(nk, kb + per);
  const __amdgpu_buffer_rsrc_t rw =
      make_rsrc(g.W + (size_t)n0 * K, (uint32_t)min(16, g.N - n0) * (uint32_t)K);
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(g.X, FUSED ? 0u : (uint32_t)g.M * (uint32_t)K);
  const int pitch = nk * 128 + 16;

  // Copies: eight lanes a row of 128 bytes, chunks turned by the row as in the tiles.
  const int cr = lane >> 3, chunk = 16 * ((lane & 7) ^ swz_row(cr));
  const int chunk8 = 16 * ((lane & 7) ^ swz_row(cr + 8));
  const uint32_t at = (uint32_t)cr * (uint32_t)K + (uint32_t)chunk;
  const uint32_t at8 = (uint32_t)(cr + 8) * (uint32_t)K + (uint32_t)chunk8;
  // steps of another wave, values past the row and rows past the last read zeros, without an
  // access of memory
  auto issue = [&](uint8_t* stage, int s) __attribute__((always_inline)) {
    uint8_t* mine = stage + wave * kStage;
    const uint32_t so = (uint32_t)min(s, nk - 1) * 128u;
    const int left = s < ke ? K - s * 128 : 0;
    const uint32_t o = chunk < left ? at : kPastEnd, o8 = chunk8 < left ? at8 : kPastEnd;
    if constexpr (XROWS >= 8) copy16(rx, mine + 2 * 1024, o, so);
    if constexpr (XROWS >= 16) copy16(rx, mine + 3 * 1024, o8, so);
    copy16(rw, mine, o, so);
    copy16(rw, mine + 1024, o8, so);
  };
  // x first: loads return in order, and the weights are many
  FusedRows rows;
  if constexpr (FUSED) rows.load(g);
#pragma unroll
  for (int u = 0; u < NS; ++u) issue(st[u], kb + u);
  if constexpr (FUSED) rows.quantize(g, xq, pitch, big, sxq);

  int4v acc = int4v{0, 0, 0, 0};
  const int r = lane & 15, c = lane >> 4;
  const int wo = r * 128 + ((c ^ swz_row(r)) << 4);
  // rows of X past the last are not kept: they repeat others
  const int xr = FUSED ? min(r, g.M - 1) : r % (XROWS ? XROWS : 1);
  const int xo = FUSED ? xr * pitch + 16 * c : 2048 + xr * 128 + ((c ^ swz_row(xr)) << 4);
  auto step = [&](uint8_t* stage, int s) __attribute__((always_inline)) {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    // this wave's copies of the step have landed: vmcnt(kCopies * (NS - 1))
    constexpr int kLeft = kCopies * (NS - 1);
    __builtin_amdgcn_s_waitcnt(0x0f70 | (kLeft & 15) | (kLeft >> 4) << 14);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    const uint8_t* mine = stage + wave * kStage;
    int4v w[2], x[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      w[h] = *reinterpret_cast<const int4v*>(mine + (wo ^ (h << 6)));
      if constexpr (FUSED)
        x[h] = *reinterpret_cast<const int4v*>(xq + xo + s * 128 + h * 64);
      else
        x[h] = *reinterpret_cast<const int4v*>(mine + (xo ^ (h << 6)));
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
      acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[h], x[h], acc, 0, 0, 0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): read before it is copied over
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    issue(stage, s + NS);
  };
  int s = kb;
  for (; s + NS <= ke; s += NS)
#pragma unroll
    for (int u = 0; u < NS; ++u) step(st[u], s + u);
#pragma unroll
  for (int u = 0; u < NS - 1; ++u)
    if (s + u < ke) step(st[u], s + u);
  __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0): no copy lands after the workgroup ends
  sums[wave][lane] = acc;
  __syncthreads();
  // lane l of a 16 x 16 result holds row l % 16 of X and four neighbouring columns
  const int m = lane & 15, n = n0 + 4 * (lane >> 4);
  if (wave != 0 || m >= g.M || n >= g.N) return;
  int4v v = sums[0][lane];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) v += sums[w][lane];
  const float sm = FUSED ? sxq[m] : g.sx[m];
  typename Val<TYPE>::T y[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = Val<TYPE>::put((float)v[e] * sm * g.sw[n + e]);
  typename Val<TYPE>::T* dst = static_cast<typename Val<TYPE>::T*>(g.Y) + (size_t)m * g.N + n;
  __builtin_memcpy(__builtin_assume_aligned(dst, sizeof(y)), y, sizeof(y));
}

template <int TYPE, int XROWS, int NS>
hipError_t launch(const StripArgs& g, hipStream_t st) {
  // N * K < 2^31 and K >= 16: at most 2^23 workgroups
  hipLaunchKernelGGL((i8_few_rows_kernel<TYPE, XROWS, NS>), dim3((unsigned)((g.N + 15) / 16)),
                     dim3(kStripThreads), 0, st, g);
  return hipGetLastError();
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

hipError_t launch_i8_strip(const int8_t* X, const float* sx, const int8_t* W, const float* sw,
                           void* Y, int type, int M, int N, int K, hipStream_t st) {
  const StripArgs g{X, nullptr, sx, W, sw, Y, M, N, K};
  hipError_t err = hipSuccess;
  i8_by_type(type, [&](auto t) {
    if (M <= 8)
      err = launch<decltype(t)::value, 8, 4>(g, st);
    else
      err = launch<decltype(t)::value, 16, 3>(g, st);
  });
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
    const StripArgs g{nullptr, x, nullptr, W, sw, y, M, N, K};
    return launch<Q4_TYPE_F32, 0, 3>(g, st);
  }
  int8_t* q = static_cast<int8_t*>(ws);
  float* s = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + p.off_s);
  const hipError_t err = launch_i8_quantize(x, Q4_TYPE_F32, q, s, M, K, st);
  if (err != hipSuccess) return err;
  return launch_i8_strip(q, s, W, sw, y, Q4_TYPE_F32, M, N, K, st);
}

}  // namespace q4
