// Row kernels of the dense feed-forward operators: what stands before and
// after the products with the Q4_0 matrices.
//
//   glu_finish       h = act(g) * u from the split-K partial sums of g and u
//   lora_shrink      t[m] = scale[id] * x[m] . A[id]^T, the adapters' narrow half (many
//                    rows; few rows: shrink_wave in the strips' launch)
//   lora_finish      y = sum of partials + t[m] . B[id]^T, the wide half
//   gradient_rows    dG = dH * U * act'(G) and dU = dH * act(G), as the fp16
//                    left operand of the gradient GEMM
//   gradient_finish  dX from the split-K partial sums
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "ffn_device.hpp"
#include "ffn_internal.hpp"
#include "q4_device.hpp"

namespace q4 {
namespace {

typedef _Float16 half4 __attribute__((ext_vector_type(4)));

constexpr int kRowThreads = 256;

__device__ __forceinline__ float bf16_to_float(uint16_t b) {
  return __builtin_bit_cast(float, (uint32_t)b << 16);
}

// ---------------------------------------------------------------------------
// Sums of split-K partials, in split order. They are bound by the round trip
// of their loads, so with SMAX > 0 (S <= SMAX) all SMAX loads are issued before
// the first addition: split indices past S - 1 repeat the last one and are not
// added. SMAX = 0 takes any S in groups of 8. V values a lane.
// ---------------------------------------------------------------------------
template <int V>
struct Vec;
template <>
struct Vec<1> {
  typedef float T;
};
template <>
struct Vec<4> {
  typedef float4v T;
};

template <int SMAX, int V>
struct Splits {
  typedef typename Vec<V>::T T;
  T t[SMAX ? SMAX : 1];
  const float* src;
  __device__ __forceinline__ void load(const float* __restrict__ at, size_t stride, int S) {
    src = at;
#pragma unroll
    for (int s = 0; s < SMAX; ++s)
      t[s] = *reinterpret_cast<const T*>(at + (size_t)min(s, S - 1) * stride);
  }
  __device__ __forceinline__ T sum(size_t stride, int S) const {
    T v{};
    if constexpr (SMAX > 0) {
#pragma unroll
      for (int s = 0; s < SMAX; ++s)
        if (s < S) v += t[s];
    } else {
      for (int s0 = 0; s0 < S; s0 += 8) {
        T p[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          p[i] = *reinterpret_cast<const T*>(src + (size_t)min(s0 + i, S - 1) * stride);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (s0 + i < S) v += p[i];
      }
    }
    return v;
  }
};

// Runs `call` with the smallest compiled SMAX for S as a compile-time number.
template <class F>
void by_splits(int S, F&& call) {
  if (S <= 2)
    call(std::integral_constant<int, 2>{});
  else if (S <= 4)
    call(std::integral_constant<int, 4>{});
  else if (S <= 8)
    call(std::integral_constant<int, 8>{});
  else if (S <= 16)
    call(std::integral_constant<int, 16>{});
  else if (S <= 32)
    call(std::integral_constant<int, 32>{});
  else if (S <= 48)
    call(std::integral_constant<int, 48>{});
  else
    call(std::integral_constant<int, 0>{});
}

// h = act(g) * u
template <int SMAX>
__global__ __launch_bounds__(64) void glu_finish_kernel(const float* __restrict__ part,
                                                        float* __restrict__ h, size_t mn, int S,
                                                        int act) {
  const size_t i = (size_t)blockIdx.x * 64 + threadIdx.x;
  if (i >= mn) return;
  Splits<SMAX, 1> g, u;
  g.load(part + i, mn, S);
  u.load(part + (size_t)S * mn + i, mn, S);
  h[i] = act_value<false>(g.sum(mn, S), act) * u.sum(mn, S);
}

template <int SMAX>
__global__ __launch_bounds__(kRowThreads) void glu_finish_f16_kernel(
    const float* __restrict__ part, _Float16* __restrict__ H, _Float16* __restrict__ G,
    _Float16* __restrict__ U, size_t mn, int S, int act) {
  const size_t i = ((size_t)blockIdx.x * kRowThreads + threadIdx.x) * 4;
  if (i >= mn) return;
  Splits<SMAX, 4> gs, us;
  gs.load(part + i, mn, S);
  us.load(part + (size_t)S * mn + i, mn, S);
  const float4v g = gs.sum(mn, S), u = us.sum(mn, S);
  half4 h, gh, uh;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    h[e] = (_Float16)(act_value<true>(g[e], act) * u[e]);
    gh[e] = (_Float16)g[e];
    uh[e] = (_Float16)u[e];
  }
  *reinterpret_cast<half4*>(H + i) = h;
  if (G) {
    *reinterpret_cast<half4*>(G + i) = gh;
    *reinterpret_cast<half4*>(U + i) = uh;
  }
}

// ---------------------------------------------------------------------------
// Adapters, narrow half, many rows, on the matrix cores (fp16 in, fp32 sums).
// A workgroup owns 64 rows of X, 32 rank indexes and one of KS shares of K; its
// 4 waves take the share's K steps of 16 in turn. For every adapter that occurs
// in the 64 rows the tile is multiplied with the 32 rows of A
// (v_mfma_f32_32x32x16_f16, both operands read straight from memory, K being
// contiguous in both) and the rows that use that adapter keep the result. Rows
// of one prompt stand together, so a tile of long prompts holds one or two
// adapters, a pass; for many short ones the passes are dealt out to `parts`
// workgroups, of which those without a pass end at once (300 rows of 100 requests,
// 576 x 2560 at rank 64, with the wide half's loads together: 91.5 -> 39.3 us a
// call). Bound by its loads: the shares keep enough of them in flight, and A is
// read once a tile (2000 rows of 11008 at rank 32 in 7 prompts: 60 us in 16-row
// tiles and one share, 29 us in eight shares, 27 us in 64-row tiles, 21 us with
// two adapters a pass). The waves'
// sums are added in wave order, the shares' by lora_rows_kernel.
// ---------------------------------------------------------------------------
constexpr int kShrinkRows = 64, kShrinkWaves = 4, kShrinkRanks = 32, kShrinkChunk = 64;

__global__ __launch_bounds__(kShrinkWaves * kWaveSize) void lora_shrink_tile_kernel(
    const _Float16* __restrict__ X, Adapters ad, float* __restrict__ tp, int M, int K, int tiles,
    int share, int shares, int parts) {
  typedef float float16v __attribute__((ext_vector_type(16)));
  __shared__ float sums[kShrinkWaves][kShrinkRows][kShrinkRanks];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tile = blockIdx.x % tiles;
  int rest = blockIdx.x / tiles;
  const int c = rest % shares;
  rest /= shares;
  const int part = rest % parts;               // of the tile's passes
  const int r0 = rest / parts * kShrinkRanks;  // first rank index
  const int m0 = tile * kShrinkRows;
  const int kb = c * share, ke = min(K, kb + share);  // multiples of a chunk
  const int R = ad.R;
  // lane l of every wave holds the adapter of row l
  int id = m0 + lane < M ? ad.ids[m0 + lane] : -1;
  if (id < 0 || id >= ad.L) id = -1;
  const int lr = lane & 31, kg = 8 * (lane >> 5);
  const _Float16* xr[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) xr[i] = X + (size_t)min(m0 + 32 * i + lr, M - 1) * K + kg;

  float16v keep[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e) keep[i][e] = 0.0f;
  unsigned long long todo = __ballot(id >= 0);
  // rows whose sums this workgroup writes: part 0 those without adapter too
  unsigned long long mine = part == 0 ? ~todo : 0;
  for (int pass = 0; todo; pass = pass + 1 == parts ? 0 : pass + 1) {
    // two adapters a pass, so that a tile across the end of a prompt reads X
    // once (a lone adapter is taken twice, its second product not kept)
    const int cur0 = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
    const unsigned long long same0 = __ballot(id == cur0);
    todo &= ~same0;
    const bool two = todo != 0;
    const int cur1 = two ? __builtin_amdgcn_readlane(id, __builtin_ctzll(todo)) : cur0;
    const unsigned long long same1 = two ? __ballot(id == cur1) : 0;
    todo &= ~same1;
    if (pass != part) continue;
    mine |= same0 | same1;
    const _Float16* ar[2];
#pragma unroll
    for (int f = 0; f < 2; ++f)  // rank indexes past R repeat the last one, not kept
      ar[f] = reinterpret_cast<const _Float16*>(ad.A) +
              ((size_t)(f ? cur1 : cur0) * R + min(r0 + lr, R - 1)) * K + kg;
    float16v acc[2][2];
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[f][i][e] = 0.0f;
    for (int k0 = kb + wave * kShrinkChunk; k0 < ke; k0 += kShrinkWaves * kShrinkChunk) {
      constexpr int kU = kShrinkChunk / 16;
      half8 xa[kU][2], b[kU][2];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          xa[u][i] = *reinterpret_cast<const half8*>(xr[i] + k0 + 16 * u);
#pragma unroll
        for (int f = 0; f < 2; ++f)
          if (f == 0 || two) b[u][f] = *reinterpret_cast<const half8*>(ar[f] + k0 + 16 * u);
      }
#pragma unroll
      for (int f = 0; f < 2; ++f)
        if (f == 0 || two)
#pragma unroll
          for (int u = 0; u < kU; ++u)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              acc[f][i] =
                  __builtin_amdgcn_mfma_f32_32x32x16_f16(xa[u][i], b[u][f], acc[f][i], 0, 0, 0);
    }
    // a 32 x 32 result: lane l holds column l % 32, register e row
    // 8 * (e / 4) + 4 * (l / 32) + e % 4
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int row = 32 * i + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3);
        keep[i][e] = (same0 >> row) & 1ull
                         ? acc[0][i][e]
                         : ((same1 >> row) & 1ull ? acc[1][i][e] : keep[i][e]);
      }
  }
  if (mine == 0) return;  // the same in every wave
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e)
      sums[wave][32 * i + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3)][lr] = keep[i][e];
  __syncthreads();
  for (int i = threadIdx.x; i < kShrinkRows * kShrinkRanks; i += kShrinkWaves * kWaveSize) {
    const int row = i / kShrinkRanks, r = i % kShrinkRanks;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kShrinkWaves; ++w) v += sums[w][row][r];
    if ((mine >> row) & 1ull && m0 + row < M && r0 + r < R)
      tp[((size_t)c * M + m0 + row) * R + r0 + r] = v;
  }
}

// One wave a row: the shares of t[m] added in order. With t16: the row scaled
// by a power of two to a largest value in [1, 2), as the fp16 operand of the
// wide half, and ts[m] = scale[id] / that power; else t[m] times scale[id].
__global__ __launch_bounds__(kRowThreads) void lora_rows_kernel(const float* __restrict__ tp,
                                                                Adapters ad,
                                                                float* __restrict__ t,
                                                                _Float16* __restrict__ t16,
                                                                float* __restrict__ ts, int M,
                                                                int KS) {
  const int lane = threadIdx.x & 63;
  const int m = blockIdx.x * (kRowThreads / kWaveSize) + (threadIdx.x >> 6);
  if (m >= M) return;
  const int R = ad.R;
  const int id = ad.ids[m];
  const bool live = id >= 0 && id < ad.L;
  const float sc = live ? ad.scale[id] : 0.0f;
  float v[2], big = 0.0f;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = lane + 64 * h;
    v[h] = r < R && live ? sum_strided(tp + (size_t)m * R + r, (size_t)M * R, KS) : 0.0f;
    big = fmaxf(big, fabsf(v[h]));
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor(big, o));
  // big in [2^e, 2^(e+1)); infinities and NaN stay what they are under any factor
  const int e = big > 0.0f ? max(-126, min(127, ilogbf(big))) : 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = lane + 64 * h;
    if (r >= R) continue;
    if (t16)
      t16[(size_t)m * R + r] = (_Float16)ldexpf(v[h], -e);
    else
      t[(size_t)m * R + r] = live ? v[h] * sc : 0.0f;
  }
  if (t16 && lane == 0) ts[m] = ldexpf(sc, e);
}

// ---------------------------------------------------------------------------
// Adapters, wide half beside split-K partial sums: one output a lane, R fp32
// multiply-adds on the fp16 row B[id][n] (16-byte loads, the first four issued
// with the partials).
// ---------------------------------------------------------------------------
template <int SMAX, class Y>
__global__ __launch_bounds__(64) void lora_finish_kernel(const float* __restrict__ part,
                                                         const float* __restrict__ t, Adapters ad,
                                                         Y* __restrict__ y, int M, int N, int S) {
  const size_t mn = (size_t)M * N;
  const size_t i = (size_t)blockIdx.x * 64 + threadIdx.x;
  if (i >= mn) return;
  Splits<SMAX, 1> p;
  p.load(part + i, mn, S);
  const int m = (int)(i / N);
  const int n = (int)(i - (size_t)m * N);
  const int id = ad.ids[m];
  float a = 0.0f;
  if (id >= 0 && id < ad.L) {
    const _Float16* br = reinterpret_cast<const _Float16*>(ad.B) + ((size_t)id * N + n) * ad.R;
    const float* tr = t + (size_t)m * ad.R;
    for (int r0 = 0; r0 < ad.R; r0 += 32) {
      float bv[4][8], tv[4][8];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int r = min(r0 + 8 * u, ad.R - 8);  // past the end: read again, not added
        load8(br + r, bv[u]);
        load8(tr + r, tv[u]);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (r0 + 8 * u < ad.R)
#pragma unroll
          for (int e = 0; e < 8; ++e) a = __builtin_fmaf(tv[u][e], bv[u][e], a);
    }
  }
  y[i] = (Y)(p.sum(mn, S) + a);
}

// ---------------------------------------------------------------------------
// Left operand of the gradient GEMM. Row m of it is [dG | dU] (mats = 2) or dY
// (mats = 1), multiplied by the power of two that takes the row's largest
// value into [2^13, 2^14) and rounded to fp16: gradients span far more binades
// than fp16 has, but within one row the largest values carry the sum, and 27
// binades below them stay normal. rs[m] undoes the factor after the product.
// Groups of eight values are stored in the order 0 4 1 5 2 6 3 7, the order
// in which masking a dword of nibbles yields half pairs.
// One workgroup a row. Up to kRowHeld groups of eight a lane (12288 columns) the
// scaled values are formed once and held in registers; a longer row is gone
// through twice. Bound by its bytes: 8 B a value read and 4 B written.
// ---------------------------------------------------------------------------
constexpr int kRowHeld = 6;

template <int MATS>
__device__ __forceinline__ void gradient_group(const uint16_t* __restrict__ dH,
                                               const uint16_t* __restrict__ G,
                                               const uint16_t* __restrict__ U, size_t at, int act,
                                               float (&dg)[8], float (&du)[8]) {
  typedef uint16_t ushort8 __attribute__((ext_vector_type(8)));
  const ushort8 h = *reinterpret_cast<const ushort8*>(dH + at);
  if constexpr (MATS == 1) {
#pragma unroll
    for (int e = 0; e < 8; ++e) dg[e] = bf16_to_float(h[e]);
    return;
  }
  const half8 g = *reinterpret_cast<const half8*>(G + at);
  const half8 u = *reinterpret_cast<const half8*>(U + at);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float a, slope;
    act_value_slope((float)g[e], act, a, slope);
    const float d = bf16_to_float(h[e]);
    dg[e] = d * (float)u[e] * slope;
    du[e] = d * a;
  }
}

__device__ __forceinline__ void store_group(_Float16* p, const float (&v)[8], float s) {
  half8 o;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    o[2 * e] = (_Float16)(v[e] * s);
    o[2 * e + 1] = (_Float16)(v[e + 4] * s);
  }
  *reinterpret_cast<half8*>(p) = o;
}

// The power of two for a row whose largest value is `big`, known to one wave
// each; the same for all lanes afterwards.
__device__ __forceinline__ int row_exponent(float big, float* wave_big) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor(big, o));
  if ((threadIdx.x & 63) == 0) wave_big[threadIdx.x >> 6] = big;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kRowThreads / kWaveSize; ++w) big = fmaxf(big, wave_big[w]);
  // the factor and its inverse stay normal fp32 numbers; a row with an infinity
  // takes the smallest, so that its finite values stay finite
  return big > 0.0f ? 13 - max(-113, min(127, ilogbf(big))) : 0;
}

template <int MATS, int HELD>
__global__ __launch_bounds__(kRowThreads) void gradient_rows_kernel(
    const uint16_t* __restrict__ dH, const uint16_t* __restrict__ G,
    const uint16_t* __restrict__ U, _Float16* __restrict__ a, float* __restrict__ rs, int N,
    int act) {
  __shared__ float wave_big[kRowThreads / kWaveSize];
  constexpr int kStep = kRowThreads * 8;
  const int m = blockIdx.x;
  const size_t row = (size_t)m * N;
  const int n0 = threadIdx.x * 8;
  _Float16* ar = a + (size_t)m * MATS * N;
  float big = 0.0f;
  if constexpr (HELD > 0) {
    float dg[HELD][8], du[HELD][8];
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      if (n0 + i * kStep >= N) break;
      gradient_group<MATS>(dH, G, U, row + n0 + i * kStep, act, dg[i], du[i]);
    }
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      if (n0 + i * kStep >= N) break;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        big = fmaxf(big, fabsf(dg[i][e]));
        if constexpr (MATS == 2) big = fmaxf(big, fabsf(du[i][e]));
      }
    }
    const int e = row_exponent(big, wave_big);
    const float s = ldexpf(1.0f, e);
    if (threadIdx.x == 0) rs[m] = ldexpf(1.0f, -e);
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      const int n = n0 + i * kStep;
      if (n >= N) break;
      store_group(ar + n, dg[i], s);
      if constexpr (MATS == 2) store_group(ar + N + n, du[i], s);
    }
  } else {
    float dg[8], du[8];
    for (int n = n0; n < N; n += kStep) {
      gradient_group<MATS>(dH, G, U, row + n, act, dg, du);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        big = fmaxf(big, fabsf(dg[e]));
        if constexpr (MATS == 2) big = fmaxf(big, fabsf(du[e]));
      }
    }
    const int e = row_exponent(big, wave_big);
    const float s = ldexpf(1.0f, e);
    if (threadIdx.x == 0) rs[m] = ldexpf(1.0f, -e);
    for (int n = n0; n < N; n += kStep) {
      gradient_group<MATS>(dH, G, U, row + n, act, dg, du);
      store_group(ar + n, dg, s);
      if constexpr (MATS == 2) store_group(ar + N + n, du, s);
    }
  }
}

template <int SMAX>
__global__ __launch_bounds__(kRowThreads) void gradient_finish_kernel(
    const float* __restrict__ part, const float* __restrict__ rs, uint16_t* __restrict__ dX,
    int M, int K, int S) {
  typedef uint16_t ushort4v __attribute__((ext_vector_type(4)));
  const size_t mk = (size_t)M * K;
  const size_t i = ((size_t)blockIdx.x * kRowThreads + threadIdx.x) * 4;
  if (i >= mk) return;
  const float r = rs[i / K];
  Splits<SMAX, 4> p;
  p.load(part + i, mk, S);
  const float4v v = p.sum(mk, S);
  ushort4v o;
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = float_to_bf16(v[e] * r);
  *reinterpret_cast<ushort4v*>(dX + i) = o;
}

unsigned blocks(size_t n, int per) { return (unsigned)((n + per - 1) / per); }

}  // namespace

hipError_t launch_glu_finish(const float* part, float* h, size_t mn, int S, int act,
                             hipStream_t st) {
  by_splits(S, [&](auto n) {
    hipLaunchKernelGGL(glu_finish_kernel<decltype(n)::value>, dim3(blocks(mn, 64)), dim3(64), 0,
                       st, part, h, mn, S, act);
  });
  return hipGetLastError();
}

hipError_t launch_glu_finish_f16(const float* part, uint16_t* H, uint16_t* G, uint16_t* U,
                                 size_t mn, int S, int act, hipStream_t st) {
  by_splits(S, [&](auto n) {
    hipLaunchKernelGGL(glu_finish_f16_kernel<decltype(n)::value>, dim3(blocks(mn, 4 * kRowThreads)),
                       dim3(kRowThreads), 0, st, part, reinterpret_cast<_Float16*>(H),
                       reinterpret_cast<_Float16*>(G), reinterpret_cast<_Float16*>(U), mn, S, act);
  });
  return hipGetLastError();
}

// Shares of K: a chunk or more for every wave, about 1024 workgroups at most.
int shrink_share(int M, int K) {
  constexpr int kStep = kShrinkWaves * kShrinkChunk;
  const int tiles = (M + kShrinkRows - 1) / kShrinkRows;
  const int s = std::max(1, std::min(512 / tiles, (K + kStep - 1) / kStep));
  return ((K + s - 1) / s + kStep - 1) / kStep * kStep;
}
int shrink_shares(int M, int K) {
  const int share = shrink_share(M, K);
  return (K + share - 1) / share;
}

hipError_t launch_lora_shrink(const uint16_t* X, const Adapters& ad, float* tp, float* t,
                              uint16_t* t16, float* ts, int M, int K, hipStream_t st) {
  const int share = shrink_share(M, K), KS = shrink_shares(M, K);
  const int tiles = (M + kShrinkRows - 1) / kShrinkRows;
  const int groups = tiles * KS * ((ad.R + kShrinkRanks - 1) / kShrinkRanks);
  const int parts = std::max(1, std::min(16, 1024 / groups));
  hipLaunchKernelGGL(lora_shrink_tile_kernel, dim3((unsigned)groups * parts),
                     dim3(kShrinkWaves * kWaveSize), 0, st, reinterpret_cast<const _Float16*>(X),
                     ad, tp, M, K, tiles, share, KS, parts);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  hipLaunchKernelGGL(lora_rows_kernel, dim3(blocks(M, kRowThreads / kWaveSize)), dim3(kRowThreads),
                     0, st, tp, ad, t, reinterpret_cast<_Float16*>(t16), ts, M, KS);
  return hipGetLastError();
}

hipError_t launch_lora_finish(const float* part, const float* t, const Adapters& ad, float* y,
                              int M, int N, int S, hipStream_t st) {
  by_splits(S, [&](auto n) {
    hipLaunchKernelGGL((lora_finish_kernel<decltype(n)::value, float>),
                       dim3(blocks((size_t)M * N, 64)), dim3(64), 0, st, part, t, ad, y, M, N, S);
  });
  return hipGetLastError();
}

hipError_t launch_lora_finish_f16(const float* part, const float* t, const Adapters& ad,
                                  uint16_t* Y, int M, int N, int S, hipStream_t st) {
  by_splits(S, [&](auto n) {
    hipLaunchKernelGGL((lora_finish_kernel<decltype(n)::value, _Float16>),
                       dim3(blocks((size_t)M * N, 64)), dim3(64), 0, st, part, t, ad,
                       reinterpret_cast<_Float16*>(Y), M, N, S);
  });
  return hipGetLastError();
}

template <int MATS>
hipError_t launch_gradient_rows_t(const uint16_t* dH, const uint16_t* G, const uint16_t* U,
                                  uint16_t* a, float* rs, int M, int N, int act, hipStream_t st) {
  const int groups = (N + 8 * kRowThreads - 1) / (8 * kRowThreads);
  auto go = [&](auto held) {
    hipLaunchKernelGGL((gradient_rows_kernel<MATS, decltype(held)::value>), dim3((unsigned)M),
                       dim3(kRowThreads), 0, st, dH, G, U, reinterpret_cast<_Float16*>(a), rs, N,
                       act);
  };
  if (groups <= 1)
    go(std::integral_constant<int, 1>{});
  else if (groups <= 2)
    go(std::integral_constant<int, 2>{});
  else if (groups <= kRowHeld)
    go(std::integral_constant<int, kRowHeld>{});
  else
    go(std::integral_constant<int, 0>{});
  return hipGetLastError();
}

hipError_t launch_gradient_rows(const uint16_t* dH, const uint16_t* G, const uint16_t* U,
                                uint16_t* a, float* rs, int M, int N, int act, int mats,
                                hipStream_t st) {
  return mats == 2 ? launch_gradient_rows_t<2>(dH, G, U, a, rs, M, N, act, st)
                   : launch_gradient_rows_t<1>(dH, G, U, a, rs, M, N, act, st);
}

hipError_t launch_gradient_finish(const float* part, const float* rs, uint16_t* dX, int M, int K,
                                  int S, hipStream_t st) {
  by_splits(S, [&](auto n) {
    hipLaunchKernelGGL(gradient_finish_kernel<decltype(n)::value>,
                       dim3(blocks((size_t)M * K, 4 * kRowThreads)), dim3(kRowThreads), 0, st, part,
                       rs, dX, M, K, S);
  });
  return hipGetLastError();
}

}  // namespace q4
