// Few rows (up to 64) through one or two Q4_0 matrices of the dense feed-forward
// operators: split-K partial sums part[mats][S][M][N] in fp32.
//
// With few rows the matrices' bytes set the pace, so every wave streams weights
// from memory straight into registers, dequantizes them there and feeds the
// matrix cores (v_mfma_f32_16x16x32_f16) without passing them through LDS.
//
//   * A wave's step is 32 rows of the matrix by a strip of 128 * DW columns.
//     Lane l holds, of the 8 rows 8 * (l / 16) .. + 7, DW dwords: the 8 * DW
//     columns from 8 * DW * (l % 16) on. Those rows are the lane's k values of
//     the product's right operand, so an 8 x 8 block of nibbles becomes the
//     operands of 8 products (product c takes column c of every lane): row
//     pairs are put side by side (v_perm), then a column pair is masked out and
//     given an exponent, and the offset and the scale are applied in packed
//     halves.
//   * Odd nibbles need no shift: 0x6400 | q is 1024 + q, and 0x5400 | (q << 4)
//     is 64 + q, both exact.
//   * The lanes of a block share its scales: each loads some of the 8 rows'
//     scales and hands them over inside the quad.
//   * The waves of a workgroup take the strip's steps in turn and add their
//     sums through LDS in wave order, each for a quarter of the rows; the splits
//     are added by the kernel that finishes the operator.
//   * Exact weights: w = (q - 8) * d has up to 14 significant bits. hi =
//     fp16(w) and lo = w - hi, which fp16 holds exactly (a multiple of d's
//     last place), take a product each: the weights are not rounded.
//   * fp32 activations (decode, up to 8 rows): x is scaled by a power of two to
//     a largest value in [2^13, 2^14) for the row and the workgroup's K range,
//     and split into hi = fp16(x) and lo = fp16(x - hi); the 16 rows of the left
//     operand are the 8 his and the 8 los. What is lost is below 2^-22 of the
//     value (or 2^-38 of the row's largest), under the roundings of an fp32 sum.
//
// Bound by their loads, of 4 or 8 bytes a lane and row: without dequantizing and
// multiplying a launch takes 21.7 of 22.5 us (8 rows, two matrices of 4096 x 11008), 28
// of 30 (33 rows), 15.2 of 16.3 (8 rows, 11008 x 4096 with adapters of rank 64), 12 of
// 12.8 (48 rows, 4096 x 4096, rank 16).
#include <algorithm>
#include <type_traits>

#include "ffn_device.hpp"
#include "ffn_internal.hpp"
#include "q4_device.hpp"

namespace q4 {
namespace {

typedef uint32_t uint4v __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4;
constexpr int kStripThreads = kWaves * kWaveSize;
constexpr int kStepRows = 32;

struct StripArgs {
  const void* X;       // fp16 [M][K], K % 32 == 0, or fp32 [M][K]
  const uint8_t* W0;
  const uint8_t* W1;
  float* part;
  int M, K, N, NB;
  int T, strips;              // strips of all matrices and of one
  int base, more;             // splits: base + 1 of the first `more` strips, base of the rest
  int S, quads;               // sums a strip has room for; rounds of kWaves steps in all
  int steps;                  // of 32 rows
  int extra;                  // first workgroups: the adapters' narrow product
  Adapters ad;
  float* t;
};

template <int DW>
struct StripWeights {
  uint32_t q[8][DW];
  uint32_t d[2 * DW];  // scales this lane loads
};

// Row pair scales 2p, 2p + 1 of the lane's block, side by side. DW = 1: four
// lanes share a block, lane i of the quad loaded rows 2i and 2i + 1; DW = 2: two
// lanes, the even one loaded rows 0..3, the odd one 4..7.
template <int DW>
__device__ __forceinline__ void scale_pairs(const StripWeights<DW>& w, half2v (&d)[4]) {
  static_assert(DW == 1 || DW == 2, "lanes of a quad share blocks");
  if constexpr (DW == 2) {
    const int m0 = (int)((w.d[0] & 0xffffu) | (w.d[1] << 16));
    const int m1 = (int)((w.d[2] & 0xffffu) | (w.d[3] << 16));
    // quad_perm [0,0,2,2] and [1,1,3,3]
    d[0] = __builtin_bit_cast(half2v, __builtin_amdgcn_mov_dpp(m0, 0xa0, 0xf, 0xf, true));
    d[1] = __builtin_bit_cast(half2v, __builtin_amdgcn_mov_dpp(m1, 0xa0, 0xf, 0xf, true));
    d[2] = __builtin_bit_cast(half2v, __builtin_amdgcn_mov_dpp(m0, 0xf5, 0xf, 0xf, true));
    d[3] = __builtin_bit_cast(half2v, __builtin_amdgcn_mov_dpp(m1, 0xf5, 0xf, 0xf, true));
  } else {
    const int m = (int)((w.d[0] & 0xffffu) | (w.d[1] << 16));
    d[0] = __builtin_bit_cast(half2v, __builtin_amdgcn_mov_dpp(m, 0x00, 0xf, 0xf, true));
    d[1] = __builtin_bit_cast(half2v, __builtin_amdgcn_mov_dpp(m, 0x55, 0xf, 0xf, true));
    d[2] = __builtin_bit_cast(half2v, __builtin_amdgcn_mov_dpp(m, 0xaa, 0xf, 0xf, true));
    d[3] = __builtin_bit_cast(half2v, __builtin_amdgcn_mov_dpp(m, 0xff, 0xf, 0xf, true));
  }
}

// First row of a step. The last step of a K that is no multiple of 32 reaches
// back into the one before it, whose rows meet activations of zero there.
__device__ __forceinline__ int step_start(int step, int K) {
  return min(step * kStepRows, max(K - kStepRows, 0));
}

// Where a lane's weights lie.
template <int DW>
struct StripSource {
  __amdgpu_buffer_rsrc_t r;
  uint32_t pitch, vq, vd;  // row 0 of the lane's 8 rows in step 0; its first scale
  int row;                 // 8 * (l / 16)
  int drow;                // first of the rows whose scales this lane loads
  int K;
  __device__ __forceinline__ void init(const StripArgs& a, const uint8_t* W, int strip, int lane) {
    constexpr int kLanes = 4 / DW;  // lanes of a block
    constexpr uint32_t kOut = 0x80000000u;
    const int cg = lane & 15;
    const int blk = strip * 4 * DW + cg / kLanes;
    const int sub = cg % kLanes;
    K = a.K;
    pitch = (uint32_t)a.NB * kBlockBytes;
    r = make_rsrc(W, (uint32_t)a.K * pitch);
    row = 8 * (lane >> 4);
    // A block column past the matrix reads zeros, and so do 8 rows past a matrix of
    // fewer than 32, from kOut on: with row 0 those offsets stay below 2^32, 31 rows of
    // the widest matrix would not.
    const bool out = blk >= a.NB || row >= a.K;
    if (out) row = 0;
    vq = out ? kOut : (uint32_t)blk * kBlockBytes + 2 + 4 * DW * sub;
    vd = out ? kOut : (uint32_t)blk * kBlockBytes;
    drow = 2 * DW * sub;
  }
  __device__ __forceinline__ void load_row(StripWeights<DW>& w, int i, uint32_t o) const {
    if constexpr (DW == 2) {
      const auto v = __builtin_amdgcn_raw_buffer_load_b64(r, vq + o, 0, 0);
#pragma unroll
      for (int j = 0; j < 2; ++j) w.q[i][j] = v[j];
    } else {
      w.q[i][0] = __builtin_amdgcn_raw_buffer_load_b32(r, vq + o, 0, 0);
    }
  }
  // Offsets stay in the lane's part of the address, which the range check sees: of
  // a group of 8 rows that ends past the matrix, the rows past it read zeros.
  __device__ __forceinline__ void load(StripWeights<DW>& w, int step) const {
    constexpr int ND = 2 * DW;
    const uint32_t o = (uint32_t)(step_start(step, K) + row) * pitch;
    const uint32_t od = vd + o + (uint32_t)drow * pitch;
#pragma unroll
    for (int i = 0; i < ND; ++i)
      w.d[i] = __builtin_amdgcn_raw_buffer_load_b16(r, od + i * pitch, 0, 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) load_row(w, i, o + i * pitch);
  }
};

struct StripMasks {
  // kept in vector registers: masking and setting the exponent is one
  // instruction, which takes at most one constant from elsewhere
  uint32_t even = 0x000f000fu, odd = 0x00f000f0u;
  __device__ __forceinline__ StripMasks() { asm volatile("" : "+v"(even), "+v"(odd)); }
};

// The products of one step: acc[f][c] += A[f] x column c of the strip.
template <int RF, int DW>
__device__ __forceinline__ void strip_products(const StripWeights<DW>& w, const half8 (&A)[RF],
                                               float4v (&acc)[RF][8 * DW], const StripMasks& mk) {
  half2v d[4];
  scale_pairs<DW>(w, d);
  const half2v off_even = {(_Float16)1032.0f, (_Float16)1032.0f};
  const half2v off_odd = {(_Float16)72.0f, (_Float16)72.0f};
  // The lo products of a column follow the hi products of the next: a product's
  // sum is ready only some 30 cycles after it was issued.
  half8 low = {};
  auto add = [&](const half8& W, int n) __attribute__((always_inline)) {
#pragma unroll
    for (int f = 0; f < RF; ++f)
      acc[f][n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(A[f], W, acc[f][n], 0, 0, 0);
  };
#pragma unroll
  for (int j = 0; j < DW; ++j)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        p[i] = __builtin_amdgcn_perm(w.q[2 * i + 1][j], w.q[2 * i][j],
                                     h ? 0x07060302u : 0x05040100u);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint4v hi, lo;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t b = c >= 2 ? p[i] >> 8 : p[i];
          half2v v;
          if (c & 1)
            v = __builtin_bit_cast(half2v, (b & mk.odd) | 0x54005400u) - off_odd;
          else
            v = __builtin_bit_cast(half2v, (b & mk.even) | 0x64006400u) - off_even;
          const half2v t = v * d[i];
          hi[i] = __builtin_bit_cast(uint32_t, t);
          lo[i] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(v, d[i], -t));
        }
        const int n = 8 * j + 4 * h + c;
        add(__builtin_bit_cast(half8, hi), n);
        if (n) add(low, n - 1);
        low = __builtin_bit_cast(half8, lo);
      }
    }
  add(low, 8 * DW - 1);
}

// LDS: fp32 activations [per][64 lanes][8 halves], then (from the same start)
// the waves' sums, up to kSumRows times 16 rows at a time.
template <int RF>
constexpr int kSumRows = RF <= 2 ? RF : (RF + 1) / 2;
template <int RF, int DW>
constexpr int kSumBytes = kSumRows<RF> * kWaves * (kWaves - 1) * 2 * DW * 1024;

__device__ __forceinline__ half2v to_half2(float a, float b) {
  typedef float float2v __attribute__((ext_vector_type(2)));
  return __builtin_convertvector(float2v{a, b}, half2v);
}

// Largest of a wave, in every lane.
__device__ __forceinline__ float wave_max(float v) {
  auto dpp = [](float x, auto ctrl) __attribute__((always_inline)) {
    return __int_as_float(
        __builtin_amdgcn_mov_dpp(__float_as_int(x), decltype(ctrl)::value, 0xf, 0xf, true));
  };
  // row_ror 8, 4, 2, 1
  v = fmaxf(v, dpp(v, std::integral_constant<int, 0x128>()));
  v = fmaxf(v, dpp(v, std::integral_constant<int, 0x124>()));
  v = fmaxf(v, dpp(v, std::integral_constant<int, 0x122>()));
  v = fmaxf(v, dpp(v, std::integral_constant<int, 0x121>()));
  const auto h = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false,
                                                  false);
  v = fmaxf(__uint_as_float(h[0]), __uint_as_float(h[1]));
  const auto w = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false,
                                                  false);
  return fmaxf(__uint_as_float(w[0]), __uint_as_float(w[1]));
}

// fp32 activations of the steps [kb, ke) as operands in LDS; inv[m] undoes the
// row's factor. Wave w takes rows w, w + kWaves .., in groups of 8 values: group g of
// the row is group g % 4 of step kb + g / 4 and goes to lane 16 * (g % 4) + m
// (its lo part to m + 8). All loads of four groups a lane are issued together,
// then `between` (the first weights: loads return in order, and what this waits
// for is the activations); more groups are read again for the second pass.
template <class Between>
__device__ __forceinline__ void stage_split(const StripArgs& a, int kb, int ke, half8* xa,
                                            float* inv, Between between) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int groups = 4 * (ke - kb);
  constexpr int kU = 4, kR = 8 / kWaves;
  __amdgpu_buffer_rsrc_t r[kR];
#pragma unroll
  for (int h = 0; h < kR; ++h) {  // rows past the last read zeros
    const int m = wave + kWaves * h;
    r[h] = make_rsrc(static_cast<const float*>(a.X) + (size_t)min(m, a.M - 1) * a.K,
                     m < a.M ? (uint32_t)a.K * 4u : 0u);
  }
  auto load = [&](int g0, float(&v)[kR][kU][8]) __attribute__((always_inline)) {
#pragma unroll
    for (int h = 0; h < kR; ++h)
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int g = g0 + 64 * u;
        const int k = step_start(kb + (g >> 2), a.K) + 8 * (g & 3);
        const uint32_t o = g < groups ? (uint32_t)k * 4u : 0x80000000u;
        const auto p = __builtin_amdgcn_raw_buffer_load_b128(r[h], o, 0, 0);
        const auto q = __builtin_amdgcn_raw_buffer_load_b128(r[h], o + 16, 0, 0);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[h][u][e] = __uint_as_float(p[e]);
          v[h][u][4 + e] = __uint_as_float(q[e]);
        }
      }
  };
  float v[kR][kU][8], big[kR] = {};
  auto largest = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int h = 0; h < kR; ++h)
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int e = 0; e < 8; ++e) big[h] = fmaxf(big[h], fabsf(v[h][u][e]));
  };
  load(lane, v);
  between();
  largest();
  for (int g0 = lane + 64 * kU; g0 < groups + lane; g0 += 64 * kU) {
    load(g0, v);
    largest();
  }
  float s[kR];
#pragma unroll
  for (int h = 0; h < kR; ++h) {
    big[h] = wave_max(big[h]);
    // the factor and its inverse stay normal
    const int e = min(14 - __builtin_amdgcn_frexp_expf(big[h]), 126);
    s[h] = ldexpf(1.0f, e);
    if (lane == 0) inv[wave + kWaves * h] = ldexpf(1.0f, -e);
  }
  for (int g0 = lane; g0 < groups + lane; g0 += 64 * kU) {
    if (groups > 64 * kU) load(g0, v);  // one round: still there
#pragma unroll
    for (int h = 0; h < kR; ++h)
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int g = g0 + 64 * u;
        if (g >= groups) continue;
        const int step = kb + (g >> 2);
        const int k = step_start(step, a.K) + 8 * (g & 3);
        half8 hi, lo;
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          // rows that the step before has taken
          const float x0 = k + e >= step * kStepRows ? v[h][u][e] : 0.0f;
          const float x1 = k + e + 1 >= step * kStepRows ? v[h][u][e + 1] : 0.0f;
          const half2v q = to_half2(x0 * s[h], x1 * s[h]);
          const half2v r = to_half2(fmaf(x0, s[h], -(float)q[0]), fmaf(x1, s[h], -(float)q[1]));
          hi[e] = q[0], hi[e + 1] = q[1];
          lo[e] = r[0], lo[e + 1] = r[1];
        }
        half8* dst = xa + (size_t)(g >> 2) * 64 + 16 * (g & 3) + wave + kWaves * h;
        dst[0] = hi;
        dst[8] = lo;
      }
  }
}

template <int RF, int DW, bool F32>
__global__ __launch_bounds__(kStripThreads) void strip_kernel(StripArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ float inv[8];
  constexpr int COLS = 128 * DW;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if ((int)blockIdx.x < a.extra) {
    // Adapters' narrow product, a wave for each (row, rank index): beside the
    // strips in one launch, whose first workgroups these are.
    using T = typename std::conditional<F32, float, _Float16>::type;
    shrink_wave(static_cast<const T*>(a.X), a.ad, a.t, a.M, a.K, (int)blockIdx.x * kWaves + wave);
    return;
  }
  const int L = xcd_logical_tile((int)blockIdx.x - a.extra, (int)gridDim.x - a.extra);
  const int full = a.base * a.T;
  const int s = L < full ? L / a.T : a.base;
  const int t = L < full ? L - s * a.T : L - full;
  const int splits = a.base + (t < a.more);
  const int mat = t >= a.strips;
  const int strip = t - mat * a.strips;
  // rounds of the waves in shares that differ by one at most
  const int kb = kWaves * (int)((int64_t)s * a.quads / splits);
  const int ke = min(a.steps, kWaves * (int)((int64_t)(s + 1) * a.quads / splits));

  StripSource<DW> src;
  src.init(a, mat ? a.W1 : a.W0, strip, lane);
  constexpr int kAhead = 2;  // steps in flight
  StripWeights<DW> w[kAhead];
  auto first_weights = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) src.load(w[u], min(kb + wave + u * kWaves, ke - 1));
  };

  const half8* xa = reinterpret_cast<const half8*>(lds);
  const _Float16* xr[RF];
  half8 A[kAhead][RF];
  auto load_x = [&](half8(&dst)[RF], int step) {
#pragma unroll
    for (int f = 0; f < RF; ++f)
      dst[f] = *reinterpret_cast<const half8*>(xr[f] + (size_t)step * kStepRows);
  };
  if constexpr (F32) {
    stage_split(a, kb, ke, reinterpret_cast<half8*>(lds), inv, first_weights);
    __syncthreads();
  } else {
#pragma unroll
    for (int f = 0; f < RF; ++f)  // rows past the last repeat it, not kept
      xr[f] = static_cast<const _Float16*>(a.X) +
              (size_t)min(16 * f + (lane & 15), a.M - 1) * a.K + 8 * (lane >> 4);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) load_x(A[u], min(kb + wave + u * kWaves, ke - 1));
    first_weights();
  }

  float4v acc[RF][8 * DW];
#pragma unroll
  for (int f = 0; f < RF; ++f)
#pragma unroll
    for (int c = 0; c < 8 * DW; ++c) acc[f][c] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
  const StripMasks mk;

  int k = kb + wave;
  for (; k + (kAhead - 1) * kWaves < ke; k += kAhead * kWaves) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int step = k + u * kWaves;
      if constexpr (F32) A[u][0] = xa[(size_t)(step - kb) * 64 + lane];
      strip_products<RF, DW>(w[u], A[u], acc, mk);
      __builtin_amdgcn_sched_barrier(0);
      const int next = min(step + kAhead * kWaves, ke - 1);
      src.load(w[u], next);
      if constexpr (!F32) load_x(A[u], next);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
#pragma unroll
  for (int u = 0; u < kAhead - 1; ++u)
    if (k + u * kWaves < ke) {  // uniform
      if constexpr (F32) A[u][0] = xa[(size_t)(k + u * kWaves - kb) * 64 + lane];
      strip_products<RF, DW>(w[u], A[u], acc, mk);
    }

  // The waves' sums. A 16 x 16 result: lane l holds column l % 16, here the
  // columns 8 * DW * (l % 16) + c of product c; register e row 4 * (l / 16) + e.
  // Wave e adds registers e of all waves, in wave order: each leaves the others'
  // in LDS, [to][from][four columns][lane].
  constexpr int C4 = 2 * DW, SF = kSumRows<RF>;
  float4v* red = reinterpret_cast<float4v*>(lds);
  auto slot = [&](int to, int from, int f, int q) __attribute__((always_inline)) {
    return ((f * kWaves + to) * (kWaves - 1) + (from < to ? from : from - 1)) * C4 * 64 + q * 64 +
           lane;
  };
  float* out = a.part + ((size_t)mat * a.S + s) * a.M * a.N;
  const bool clear = splits < a.S && s == 0;  // the last sum of a strip with fewer splits
  const size_t last = (size_t)(a.S - 1) * a.M * a.N;
  const float4v zero = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int f0 = 0; f0 < RF; f0 += SF) {
    if (F32 || f0) __syncthreads();  // the activations, or the sums before, have been read
#pragma unroll
    for (int f = f0; f < f0 + SF && f < RF; ++f)
#pragma unroll
      for (int e = 0; e < kWaves; ++e) {
        if (e == wave) continue;  // uniform
#pragma unroll
        for (int q = 0; q < C4; ++q)
          red[slot(e, wave, f - f0, q)] = float4v{acc[f][4 * q][e], acc[f][4 * q + 1][e],
                                                  acc[f][4 * q + 2][e], acc[f][4 * q + 3][e]};
      }
    __syncthreads();
#pragma unroll
    for (int f = f0; f < f0 + SF && f < RF; ++f) {
      float4v v[C4];
#pragma unroll
      for (int q = 0; q < C4; ++q) {
        float4v own;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4v r = acc[f][4 * q + i];
          own[i] = wave < 2 ? (wave == 0 ? r[0] : r[1]) : (wave == 2 ? r[2] : r[3]);
        }
        v[q] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int from = 0; from < kWaves; ++from)
          v[q] += from == wave ? own : red[slot(wave, from, f - f0, q)];
      }
      const int n = strip * COLS + 8 * DW * (lane & 15);
      if constexpr (F32) {
        // rows 8 .. 15 are the lo parts of 0 .. 7: lanes of the lower half add
        // the first half of their columns, those of the upper half the second
#pragma unroll
        for (int q = 0; q < C4 / 2; ++q)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const auto h = __builtin_amdgcn_permlane32_swap(
                __float_as_uint(v[q][i]), __float_as_uint(v[q + C4 / 2][i]), false, false);
            v[q][i] = __uint_as_float(h[0]) + __uint_as_float(h[1]);
          }
        const int m = 4 * ((lane >> 4) & 1) + wave;
        if (m < a.M && n < a.N) {
          float* dst = out + (size_t)m * a.N + n + (lane >> 5) * 2 * C4;
#pragma unroll
          for (int q = 0; q < C4 / 2; ++q) {
            *reinterpret_cast<float4v*>(dst + 4 * q) = v[q] * inv[m];
            if (clear) *reinterpret_cast<float4v*>(dst + last + 4 * q) = zero;
          }
        }
      } else {
        const int m = 16 * f + 4 * (lane >> 4) + wave;
        if (m < a.M && n < a.N) {
          float* dst = out + (size_t)m * a.N + n;
#pragma unroll
          for (int q = 0; q < C4; ++q) {
            *reinterpret_cast<float4v*>(dst + 4 * q) = v[q];
            if (clear) *reinterpret_cast<float4v*>(dst + last + 4 * q) = zero;
          }
        }
      }
    }
  }
}

template <int RF, int DW, bool F32>
hipError_t launch_strip_t(const StripArgs& a, hipStream_t st) {
  int lds = kSumBytes<RF, DW>;
  if (F32) lds = std::max(lds, (a.quads + a.base - 1) / a.base * kWaves * 1024);
  hipLaunchKernelGGL((strip_kernel<RF, DW, F32>), dim3(a.extra + a.base * a.T + a.more),
                     dim3(kStripThreads), lds, st, a);
  return hipGetLastError();
}

}  // namespace

// Strip width: two dwords a lane for decode (rows of 144 bytes, 64 accumulator
// registers), one for up to 64 rows (128 accumulator registers at 64 rows).
//
// Splits: any number of workgroups G can be shared out over the strips, some of
// which then have one split more than the rest; tried are equal splits and one
// to four workgroups a CU. A CU's time is its share of all rounds of steps (a
// round: a step of each wave), but at least the longest workgroup's, which alone
// on a CU takes longer for a round, plus about 2 us a workgroup for staging and
// sums, plus the partial sums, written and read again. Measured (decode, 8 rows):
// two matrices of 4096 x 11008 (86 strips) with G = 172, 256, 512, 768, 1024:
// 24.5, 23.2, 20.9, 22.2, 24.3 us; one of 11008 x 4096 (16 strips) with 128, 192,
// 256, 512, 768: 17.5, 16.4, 15.0, 16.7, 20.5 us. fp16, 33 rows, two of 4096 x
// 11008 (172 strips) with 256, 344, 512, 688, 768: 34.4, 29.8, 27.1, 27.7, 28.5.
StripPlan plan_strip(int M, int N, int K, int mats, bool f32) {
  StripPlan p{};
  p.DW = f32 ? 2 : 1;
  p.strips = (N + 128 * p.DW - 1) / (128 * p.DW);
  p.steps = (K + kStepRows - 1) / kStepRows;
  const int quads = (p.steps + kWaves - 1) / kWaves;
  const int T = mats * p.strips;
  // 128 KiB of staged activations at most
  const int least = f32 ? (quads + 31) / 32 : 1;
  const double unit[2] = {f32 ? 0.95 : 0.8, f32 ? 0.6 : 0.5};  // us
  const double sums = 8.0 * mats * (double)M * N / 4e6;  // us a split
  double best = 1e30;
  auto consider = [&](long long G) {
    const int base = (int)(G / T), more = (int)(G % T), S = base + (more > 0);
    if (base < least || S > quads) return;
    const double n = (double)((G + 255) / 256);
    const double longest = unit[0] * ((quads + base - 1) / base);
    const double shared = unit[1] * n * T * quads / G;
    const double cost = std::max(longest, shared) + 2.0 * n + sums * S;
    if (cost < best) {
      best = cost;
      p.base = base;
      p.more = more;
      p.S = S;
    }
  };
  for (int s = least; s <= std::max(least, std::min(quads, 64)); ++s) consider((long long)T * s);
  for (int r = 1; r <= 4; ++r) consider(256 * r);
  p.part_bytes = (size_t)mats * p.S * M * N * sizeof(float);
  return p;
}

hipError_t launch_strip(const void* X, const uint8_t* W0, const uint8_t* W1, float* part, int M,
                        int N, int K, bool f32, const StripPlan& p, hipStream_t st,
                        const Adapters* ad, float* t) {
  StripArgs a{};
  a.X = X;
  a.W0 = W0;
  a.W1 = W1;
  a.part = part;
  a.M = M;
  a.K = K;
  a.N = N;
  a.NB = N / kBlockWeights;
  a.strips = p.strips;
  a.T = (W1 ? 2 : 1) * p.strips;
  a.base = p.base;
  a.more = p.more;
  a.S = p.S;
  a.steps = p.steps;
  a.quads = (p.steps + kWaves - 1) / kWaves;
  if (ad) {
    a.ad = *ad;
    a.t = t;
    // a multiple of the XCDs, so that the strips' workgroups keep theirs
    a.extra = ((M * ad->R + kWaves - 1) / kWaves + kNumXcd - 1) / kNumXcd * kNumXcd;
  }
  if (f32) return launch_strip_t<1, 2, true>(a, st);
  switch ((M + 15) / 16) {
    case 1: return launch_strip_t<1, 1, false>(a, st);
    case 2: return launch_strip_t<2, 1, false>(a, st);
    case 3: return launch_strip_t<3, 1, false>(a, st);
    case 4: return launch_strip_t<4, 1, false>(a, st);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace q4
