// Weights' gradient of up to 16 output channels (the rank of an adapter):
//   dW[n][k] = sum_m (dY[m][n] * sx[m]) * X[m][k]
// in one kernel. dY is little and X is much: a workgroup owns 64 columns of X, whose rows are on
// their way into LDS while it makes its left operand: all of dY * sx, scaled column by column
// and rounded to fp16 as for the tiles, transposed in LDS. Its waves then share out the rows:
// each multiplies steps of 32 by v_mfma_f32_16x16x32_f16, copied memory -> LDS several steps
// ahead into a part of its own, and their sums meet in LDS, in the order of the waves.
//
// Up to 2048 rows (4096 of eight channels) fit a workgroup of eight waves; more are split over
// workgroups of four waves and half as many rows, two of which fit a CU. Each split scales by
// the power of two of its own rows and takes it back (exact), so splits are sums of their own,
// added in their order by a second kernel.
//
// What bounds it: rank 16 of 1999 rows of 11008 9.3 us, of which X takes 4.4 at a large copy's
// rate; the rest is the start, dY's way from memory and its 32768 values' conversion (a
// microsecond on a CU's four units), which the copies in flight only hide as far as they fit
// LDS. By a transposing kernel and the tiles: 15.8. Rank 16 of 8192 rows of 4096 12.9 us by four
// waves, 12.7 by eight, of 11008 27.8 and 29.2 (tiles 20.3 and 29.8), of 4096 rows of 4096 9.5
// and 10.7 (14.6); of a row 5.3 (6.5). Past 64 splits the tiles take over.
#include <algorithm>

#include "i8_device.hpp"
#include "i8_internal.hpp"
#include "i8_tile.hpp"

namespace q4 {
namespace {


constexpr int kCols = 64;               // of X, a workgroup
constexpr int kStepRows = 32;           // of X, a step of a wave
constexpr int kStepCopy = kStepRows * kCols;
constexpr int NS = 5;                   // steps of a wave in LDS
constexpr int kWaveValues = 4096;       // of dY in LDS, a wave
constexpr int kMaxSplits = 64;

struct ChannelArgs {
  const uint16_t* dY;
  const float* sx;
  const int8_t* X;
  uint16_t* dW;
  float* part;  // fp32 [S][N][K]
  int M, K, tiles, S, chunk;
};

// Where the 16-byte chunk c of a step's row k stands: c ^ swz_step(k). The rows that 32 lanes
// read at once, 16 of one chunk, meet no bank twice.
__device__ __forceinline__ int swz_step(int k) { return 2 * ((k >> 2) & 1) + ((k >> 3) & 1); }

// N: output channels, 8 or 16
template <int N, int kWaves>
__global__ __launch_bounds__(kWaves* kWaveSize) void i8_few_channels_kernel(ChannelArgs g) {
  constexpr int kThreads = kWaves * kWaveSize;
  constexpr int kRows = kWaves * kWaveValues / N;  // of dY
  constexpr int kPitch = kRows * 2 + 16;  // bytes of a channel in LDS
  constexpr int kPieces = N / 8;          // of a row of dY
  constexpr int kLanes = kThreads / kPieces;
  constexpr int P = kRows / 2 / kLanes;   // pairs of rows of a lane
  __shared__ __attribute__((aligned(16))) uint8_t a[N * kPitch];
  __shared__ uint32_t big[kWaves][N];
  __shared__ float up[N], down[N];
  // The steps' stages are apart, so that the compiler can tell a copy into one from a read of
  // another; in each every wave has its own part.
  __shared__ __attribute__((aligned(1024))) uint8_t s0[kWaves * kStepCopy], s1[kWaves * kStepCopy],
      s2[kWaves * kStepCopy], s3[kWaves * kStepCopy], s4[kWaves * kStepCopy];
  uint8_t* const st[NS] = {s0, s1, s2, s3, s4};
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  // neighbours, which share the lines of X, on one XCD
  const int L = xcd_logical_tile(blockIdx.x, gridDim.x);
  const int sp = L / g.tiles, j0 = (L - sp * g.tiles) * kCols;
  const int m0 = sp * g.chunk, left = min(g.M - m0, g.chunk);  // at least one, at most kRows
  const int nk = (left + kStepRows - 1) / kStepRows, per = (nk + kWaves - 1) / kWaves;
  const int kb = min(nk, wave * per), ke = min(nk, kb + per);

  // dY first: loads return in order, and X is much. A lane takes pairs of neighbouring rows,
  // eight columns of each.
  const int half = t % kPieces, pair = t / kPieces;
  Piece<Q4_TYPE_BF16> v[P][2];
  float s[P][2];
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int m = m0 + min(2 * (p * kLanes + pair) + h, left - 1);
      v[p][h].load(g.dY + (size_t)m * N + 8 * half);
      s[p][h] = g.sx[m];
    }
  asm volatile("" ::: "memory");  // the copies below stay below
  __builtin_amdgcn_sched_barrier(0);

  // Copies: four lanes a row of 64 bytes. Rows past M are past the end and become zeros, rows
  // of the next split meet zeros of dY, columns past K are not kept; steps past the last copy
  // zeros, without an access of memory, and are not read.
  const __amdgpu_buffer_rsrc_t rx =
      make_rsrc(g.X + j0, (uint32_t)g.M * (uint32_t)g.K - (uint32_t)j0);
  const uint32_t at = (uint32_t)(lane >> 2) * (uint32_t)g.K +
                      16u * (uint32_t)((lane & 3) ^ swz_step(lane >> 2));
  auto issue = [&](uint8_t* stage, int k) __attribute__((always_inline)) {
    uint8_t* mine = stage + wave * kStepCopy;
    const uint32_t so = (uint32_t)(m0 + min(k, nk - 1) * kStepRows) * (uint32_t)g.K;
    copy16(rx, mine, k < ke ? at : kPastEnd, so);
    copy16(rx, mine + kStepCopy / 2, k < ke ? at + 16u * (uint32_t)g.K : kPastEnd, so);
  };
#pragma unroll
  for (int u = 0; u < NS; ++u) issue(st[u], kb + u);

  // Rows past the last are the last times zero: zeros, or a NaN in a channel that holds an
  // infinity or a NaN there and so has no finite result. fmaxf passes over NaN: what a channel
  // with one is scaled by does not matter.
  float x[P][2][8];
  float largest[8] = {};
#pragma unroll
  for (int p = 0; p < P; ++p)
    if (2 * p * kLanes < left) {  // uniform
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (2 * (p * kLanes + pair) + h >= left) s[p][h] = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
#pragma unroll
        for (int h = 0; h < 2; ++h) x[p][h][e] = v[p][h][e] * s[p][h];
        largest[e] = fmaxf(fmaxf(largest[e], fabsf(x[p][0][e])), fabsf(x[p][1][e]));
      }
    }
  uint32_t most[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) most[e] = magnitude(largest[e]);
  const int col = wave_max_of_eight<kPieces>(most);
  if (lane < N) big[wave][8 * half + col] = most[0];
  lds_only_barrier();
  if (t < N) {
    uint32_t b = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) b = max(b, big[w][t]);
    const PowerOfTwo f = to_fp16_range(b);
    up[t] = f.up;
    down[t] = f.down;
  }
  lds_only_barrier();
#pragma unroll
  for (int p = 0; p < P; ++p)
    if (2 * p * kLanes < left)  // and so all rows of the last step
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float f = up[8 * half + e];
        *reinterpret_cast<half2v*>(a + (8 * half + e) * kPitch + 4 * (p * kLanes + pair)) =
            half2v{(_Float16)(x[p][0][e] * f), (_Float16)(x[p][1][e] * f)};
      }
  lds_only_barrier();

  float4v acc[kCols / 16];
#pragma unroll
  for (int j = 0; j < kCols / 16; ++j) acc[j] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
  // Lane l takes channel l % 16 and rows 8 * (l / 16) .. of a step; of eight channels the upper
  // lanes repeat the lower and are not kept.
  const uint8_t* ar = a + (lane & (N - 1)) * kPitch + 16 * (lane >> 4);
  const int kr = 8 * (lane >> 4) + ((lane & 15) >> 1);
  const int bo = wave * kStepCopy + kr * kCols + 8 * (lane & 1), bs = swz_step(kr);
  auto step = [&](uint8_t* stage, int k) __attribute__((always_inline)) {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    // this wave's copies of the step have landed: vmcnt(2 * (NS - 1))
    constexpr int kLeft = 2 * (NS - 1);
    __builtin_amdgcn_s_waitcnt(0x0f70 | (kLeft & 15) | (kLeft >> 4) << 14);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    const half8 x = *reinterpret_cast<const half8*>(ar + k * (2 * kStepRows));
    int2v b[kCols / 16];
#pragma unroll
    for (int j = 0; j < kCols / 16; ++j)
      b[j] = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
          (__attribute__((address_space(3))) int2v*)(stage + bo + ((j ^ bs) << 4)));
#pragma unroll
    for (int j = 0; j < kCols / 16; ++j)
      acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(to_halves(b[j]), x, acc[j], 0, 0, 0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): read before it is copied over
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    issue(stage, k + NS);
  };
  int k = kb;
  for (; k + NS <= ke; k += NS)
#pragma unroll
    for (int u = 0; u < NS; ++u) step(st[u], k + u);
#pragma unroll
  for (int u = 0; u < NS - 1; ++u)
    if (k + u < ke) step(st[u], k + u);
  __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0): no copy lands after the workgroup ends

  // lane l of a 16 x 16 result holds channel l % 16 and four neighbouring columns
  float4v* sums = reinterpret_cast<float4v*>(a);
  static_assert(kWaves * kCols / 16 * kWaveSize * 16 <= N * kPitch, "sums fit");
  __syncthreads();  // `a` has been read
#pragma unroll
  for (int j = 0; j < kCols / 16; ++j) sums[(wave * (kCols / 16) + j) * kWaveSize + lane] = acc[j];
  __syncthreads();
  const int n = lane & 15, c = j0 + 16 * wave + 4 * (lane >> 4);
  if (wave >= kCols / 16 || n >= N || c >= g.K) return;
  float4v sum = sums[wave * kWaveSize + lane];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) sum += sums[(w * (kCols / 16) + wave) * kWaveSize + lane];
  sum *= down[n];
  if (g.S > 1) {
    *reinterpret_cast<float4v*>(g.part + ((size_t)sp * N + n) * g.K + c) = sum;
    return;
  }
  uint32_t y[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = i8_to_bf16(sum[e]);
  *reinterpret_cast<uint2*>(g.dW + (size_t)n * g.K + c) =
      make_uint2(y[0] | (y[1] << 16), y[2] | (y[3] << 16));
}

template <int N, int WAVES>
void launch(const ChannelArgs& g, hipStream_t st) {
  hipLaunchKernelGGL((i8_few_channels_kernel<N, WAVES>), dim3((unsigned)(g.tiles * g.S)),
                     dim3(WAVES * kWaveSize), 0, st, g);
}

}  // namespace

bool plan_i8_few_channels(I8Plan& p, int M, int N, int K) {
  if (N > 16) return false;
  const int most = 4 * kWaveValues / N;
  if (M > kMaxSplits * most) return false;
  const int S = M <= 2 * most ? 1 : (M + most - 1) / most;
  p.strip = true;
  p.kper = ((M + S - 1) / S + 63) / 64;  // of 64 rows, at most what a workgroup takes
  p.S = (M + p.kper * 64 - 1) / (p.kper * 64);
  if (p.S > 1) p.ws_bytes = (size_t)p.S * N * K * sizeof(float);
  return true;
}

hipError_t launch_i8_few_channels(const uint16_t* dY, const int8_t* X, const float* sx,
                                  uint16_t* dW, int M, int N, int K, float* part, const I8Plan& p,
                                  hipStream_t st) {
  const ChannelArgs g{dY, sx, X, dW, part, M, K, (K + kCols - 1) / kCols, p.S, p.kper * 64};
  if (N == 8)
    p.S == 1 ? launch<8, 8>(g, st) : launch<8, 4>(g, st);
  else
    p.S == 1 ? launch<16, 8>(g, st) : launch<16, 4>(g, st);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || p.S == 1) return err;
  return launch_i8_gradient_finish(part, nullptr, dW, N, K, p.S, st);
}

}  // namespace q4
