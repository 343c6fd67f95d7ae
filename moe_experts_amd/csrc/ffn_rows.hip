// Row kernels of the dense feed-forward operators: what stands before and
// after the products with the Q4_0 matrices.
//
//   glu_finish       h = act(g) * u from the split-K partial sums of g and u
//   lora_shrink      t[m] = scale[id] * x[m] . A[id]^T, the adapters' narrow half
//   lora_finish      y = sum of partials + t[m] . B[id]^T, the wide half
//   gradient_rows    dG = dH * U * act'(G) and dU = dH * act(G), as the fp16
//                    left operand of the gradient GEMM
//   gradient_finish  dX from the split-K partial sums
#include <hip/hip_runtime.h>

#include "ffn_act.hpp"
#include "ffn_internal.hpp"
#include "q4_device.hpp"

namespace q4 {
namespace {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half4 __attribute__((ext_vector_type(4)));
typedef float float4v __attribute__((ext_vector_type(4)));

constexpr int kRowThreads = 256;

__device__ __forceinline__ float bf16_to_float(uint16_t b) {
  return __builtin_bit_cast(float, (uint32_t)b << 16);
}

// fp32 -> bf16, to nearest, ties to even; a NaN stays one (its high bits with
// the quiet bit set).
__device__ __forceinline__ uint16_t float_to_bf16(float f) {
  const uint32_t u = __builtin_bit_cast(uint32_t, f);
  if ((u & 0x7fffffffu) > 0x7f800000u) return (uint16_t)((u >> 16) | 0x40u);
  return (uint16_t)((u + 0x7fffu + ((u >> 16) & 1u)) >> 16);
}

// ---------------------------------------------------------------------------
// h = act(g) * u, four consecutive values a lane, both sums in split order.
// Bound by the round trip of its loads: all of one group of splits are issued
// before the first addition.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float4v sum_splits4(const float* __restrict__ src, size_t stride,
                                               int S) {
  float4v v = {0.0f, 0.0f, 0.0f, 0.0f};
  int s = 0;
  for (; s + 4 <= S; s += 4) {
    float4v t[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      t[i] = *reinterpret_cast<const float4v*>(src + (size_t)(s + i) * stride);
#pragma unroll
    for (int i = 0; i < 4; ++i) v += t[i];
  }
  for (; s < S; ++s) v += *reinterpret_cast<const float4v*>(src + (size_t)s * stride);
  return v;
}

__global__ __launch_bounds__(64) void glu_finish_kernel(const float* __restrict__ part,
                                                        float* __restrict__ h, size_t mn, int S,
                                                        int act) {
  const size_t i = (size_t)blockIdx.x * 64 + threadIdx.x;
  if (i >= mn) return;
  const float g = sum_strided(part + i, mn, S);
  const float u = sum_strided(part + (size_t)S * mn + i, mn, S);
  h[i] = act_value(g, act) * u;
}

__global__ __launch_bounds__(kRowThreads) void glu_finish_f16_kernel(
    const float* __restrict__ part, _Float16* __restrict__ H, _Float16* __restrict__ G,
    _Float16* __restrict__ U, size_t mn, int S, int act) {
  const size_t i = ((size_t)blockIdx.x * kRowThreads + threadIdx.x) * 4;
  if (i >= mn) return;
  const float4v g = sum_splits4(part + i, mn, S);
  const float4v u = sum_splits4(part + (size_t)S * mn + i, mn, S);
  half4 h, gh, uh;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    h[e] = (_Float16)(act_value(g[e], act) * u[e]);
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
// Adapters, narrow half, few rows: one wave per (row m, rank index r) runs one
// dot product of K, eight values a lane and step; the lanes are added by a
// fixed butterfly. Every adapter row is read once for every row of x that uses
// it (16-byte loads), so this form is for rows that mostly use different
// adapters. A row without adapter gets zeros.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4v a = *reinterpret_cast<const float4v*>(p);
  const float4v b = *reinterpret_cast<const float4v*>(p + 4);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[e] = a[e];
    v[4 + e] = b[e];
  }
}
__device__ __forceinline__ void load8(const _Float16* p, float (&v)[8]) {
  const half8 a = *reinterpret_cast<const half8*>(p);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = (float)a[e];
}

template <class X>
__device__ __forceinline__ void shrink_wave(const X* __restrict__ x, const Adapters& ad,
                                            float* __restrict__ t, int M, int K, int w) {
  const int lane = threadIdx.x & 63;
  const int m = w / ad.R;
  if (m >= M) return;
  const int r = w - m * ad.R;
  const int id = ad.ids[m];
  float sum = 0.0f;
  if (id >= 0 && id < ad.L) {
    const X* xr = x + (size_t)m * K;
    const _Float16* ar = reinterpret_cast<const _Float16*>(ad.A) + ((size_t)id * ad.R + r) * K;
    constexpr int kStep = 64 * 8, kUnroll = 4;
    for (int k0 = lane * 8; k0 < K; k0 += kStep * kUnroll) {
      float xv[kUnroll][8], av[kUnroll][8];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        // past the end the last group is read again and not added
        const int k = min(k0 + u * kStep, K - 8);
        load8(xr + k, xv[u]);
        load8(ar + k, av[u]);
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (k0 + u * kStep < K)
#pragma unroll
          for (int e = 0; e < 8; ++e) sum = __builtin_fmaf(xv[u][e], av[u][e], sum);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
    sum *= ad.scale[id];
  }
  if (lane == 0) t[(size_t)m * ad.R + r] = sum;
}

template <class X>
__global__ __launch_bounds__(kRowThreads) void lora_shrink_kernel(const X* __restrict__ x,
                                                                  Adapters ad,
                                                                  float* __restrict__ t, int M,
                                                                  int K) {
  shrink_wave(x, ad, t, M, K, blockIdx.x * (kRowThreads / kWaveSize) + threadIdx.x / kWaveSize);
}

// ---------------------------------------------------------------------------
// Adapters, narrow half, many rows, on the matrix cores (fp16 in, fp32 sums).
// A workgroup owns 16 rows of X and the whole of K; its 8 waves take K steps
// of 32 in turn. For every adapter that occurs in the 16 rows the tile is
// multiplied with all R rows of A (v_mfma_f32_16x16x32_f16, both operands read
// straight from memory, K being contiguous in both) and the rows that use that
// adapter keep the result. Rows of one prompt stand together, so a tile nearly
// always holds one or two adapters. The waves' sums are added in wave order.
// With t16: rows scaled by a power of two to a largest value in [1, 2), as the
// fp16 operand of the wide half, and ts[m] = scale[id] / that power.
// ---------------------------------------------------------------------------
constexpr int kShrinkRows = 16, kShrinkWaves = 8;
constexpr int kMaxR = Q4_LORA_MAX_R;

__global__ __launch_bounds__(kShrinkWaves * kWaveSize) void lora_shrink_tile_kernel(
    const _Float16* __restrict__ X, Adapters ad, float* __restrict__ t,
    _Float16* __restrict__ t16, float* __restrict__ ts, int M, int K) {
  __shared__ __attribute__((aligned(16))) float sums[kShrinkWaves][kShrinkRows][kMaxR];
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int m0 = blockIdx.x * kShrinkRows;
  const int R = ad.R;
  // lane l of every wave holds the adapter of row l % 16
  const int row = lane & 15;
  int id = m0 + row < M ? ad.ids[m0 + row] : -1;
  if (id < 0 || id >= ad.L) id = -1;
  for (int i = lane; i < kShrinkRows * R; i += kWaveSize) sums[wave][i / R][i % R] = 0.0f;

  const _Float16* xr = X + (size_t)min(m0 + row, M - 1) * K + 8 * (lane >> 4);
  unsigned todo = (unsigned)__ballot(id >= 0) & 0xffffu;
  while (todo) {
    const int cur = __builtin_amdgcn_readlane(id, __builtin_ctz(todo));
    const unsigned same = (unsigned)__ballot(id == cur) & 0xffffu;
    todo &= ~same;
    // 32 rows of A at a time
    for (int r0 = 0; r0 < R; r0 += 32) {
      const _Float16* ar[2];
#pragma unroll
      for (int f = 0; f < 2; ++f)  // rank indexes past R repeat the last one, not kept
        ar[f] = reinterpret_cast<const _Float16*>(ad.A) +
                ((size_t)cur * R + min(r0 + 16 * f + row, R - 1)) * K + 8 * (lane >> 4);
      float4v acc[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
      constexpr int kU = 4;  // K steps in flight
      for (int k0 = wave * 32; k0 < K; k0 += kU * kShrinkWaves * 32) {
        half8 xa[kU], b[kU][2];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int k = k0 + u * kShrinkWaves * 32;
          const int kc = min(k, K - 32);
          xa[u] = *reinterpret_cast<const half8*>(xr + kc);
#pragma unroll
          for (int f = 0; f < 2; ++f) b[u][f] = *reinterpret_cast<const half8*>(ar[f] + kc);
        }
#pragma unroll
        for (int u = 0; u < kU; ++u)
          if (k0 + u * kShrinkWaves * 32 < K)
#pragma unroll
            for (int f = 0; f < 2; ++f)
              acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_f16(xa[u], b[u][f], acc[f], 0, 0, 0);
      }
      // a 16 x 16 result: lane l holds column l % 16, register e row 4 * (l / 16) + e
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const int r = r0 + 16 * f + row;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int mr = 4 * (lane >> 4) + e;
          if (r < R && ((same >> mr) & 1u)) sums[wave][mr][r] = acc[f][e];
        }
      }
    }
  }
  __syncthreads();
  // each wave finishes two rows: lane l takes r = l and l + 64
#pragma unroll
  for (int i = 0; i < kShrinkRows / kShrinkWaves; ++i) {
    const int mr = wave + i * kShrinkWaves;
    const int m = m0 + mr;
    if (m >= M) continue;
    const int mid = __builtin_amdgcn_readlane(id, mr);
    const float sc = mid >= 0 ? ad.scale[mid] : 0.0f;
    float v[2], big = 0.0f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = lane + 64 * h;
      v[h] = 0.0f;
      if (r < R && mid >= 0)
        for (int w = 0; w < kShrinkWaves; ++w) v[h] += sums[w][mr][r];
      big = fmaxf(big, fabsf(v[h]));
    }
    if (t16) {
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor(big, o));
      // big in [2^e, 2^(e+1)); infinities and NaN stay what they are under any factor
      const int e = big > 0.0f ? max(-126, min(127, ilogbf(big))) : 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = lane + 64 * h;
        if (r < R) t16[(size_t)m * R + r] = (_Float16)ldexpf(v[h], -e);
      }
      if (lane == 0) ts[m] = ldexpf(sc, e);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = lane + 64 * h;
        if (r < R) t[(size_t)m * R + r] = mid >= 0 ? v[h] * sc : 0.0f;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Adapters, wide half beside split-K partial sums: one output a lane, R fp32
// multiply-adds on the fp16 row B[id][n] (16-byte loads).
// ---------------------------------------------------------------------------
template <class Y>
__global__ __launch_bounds__(64) void lora_finish_kernel(const float* __restrict__ part,
                                                         const float* __restrict__ t, Adapters ad,
                                                         Y* __restrict__ y, int M, int N, int S) {
  const size_t mn = (size_t)M * N;
  const size_t i = (size_t)blockIdx.x * 64 + threadIdx.x;
  if (i >= mn) return;
  const int m = (int)(i / N);
  const int n = (int)(i - (size_t)m * N);
  const int id = ad.ids[m];
  const float v = sum_strided(part + i, mn, S);
  float a = 0.0f;
  if (id >= 0 && id < ad.L) {
    const _Float16* br = reinterpret_cast<const _Float16*>(ad.B) + ((size_t)id * N + n) * ad.R;
    const float* tr = t + (size_t)m * ad.R;
    for (int r = 0; r < ad.R; r += 8) {
      float bv[8], tv[8];
      load8(br + r, bv);
      load8(tr + r, tv);
#pragma unroll
      for (int e = 0; e < 8; ++e) a = __builtin_fmaf(tv[e], bv[e], a);
    }
  }
  y[i] = (Y)(v + a);
}

// ---------------------------------------------------------------------------
// Left operand of the gradient GEMM. Row m of it is [dG | dU] (mats = 2) or dY
// (mats = 1), multiplied by the power of two that takes the row's largest
// value into [2^13, 2^14) and rounded to fp16: gradients span far more binades
// than fp16 has, but within one row the largest values carry the sum, and 27
// binades below them stay normal. rs[m] undoes the factor after the product.
// Groups of eight values are stored in the order 0 4 1 5 2 6 3 7, the order
// in which masking a dword of nibbles yields half pairs.
// One workgroup a row, two passes over it (the second from L2).
// ---------------------------------------------------------------------------
__device__ __forceinline__ void gradient_group(const uint16_t* __restrict__ dH,
                                               const uint16_t* __restrict__ G,
                                               const uint16_t* __restrict__ U, size_t at, int act,
                                               int mats, float (&dg)[8], float (&du)[8]) {
  typedef uint16_t ushort8 __attribute__((ext_vector_type(8)));
  const ushort8 h = *reinterpret_cast<const ushort8*>(dH + at);
  if (mats == 1) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      dg[e] = bf16_to_float(h[e]);
      du[e] = 0.0f;
    }
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

__global__ __launch_bounds__(kRowThreads) void gradient_rows_kernel(
    const uint16_t* __restrict__ dH, const uint16_t* __restrict__ G,
    const uint16_t* __restrict__ U, _Float16* __restrict__ a, float* __restrict__ rs, int N,
    int act, int mats) {
  __shared__ float wave_big[kRowThreads / kWaveSize];
  const int m = blockIdx.x;
  const size_t row = (size_t)m * N;
  float big = 0.0f;
  for (int n = threadIdx.x * 8; n < N; n += kRowThreads * 8) {
    float dg[8], du[8];
    gradient_group(dH, G, U, row + n, act, mats, dg, du);
#pragma unroll
    for (int e = 0; e < 8; ++e) big = fmaxf(big, fmaxf(fabsf(dg[e]), fabsf(du[e])));
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor(big, o));
  if ((threadIdx.x & 63) == 0) wave_big[threadIdx.x >> 6] = big;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kRowThreads / kWaveSize; ++w) big = fmaxf(big, wave_big[w]);
  // the factor and its inverse stay normal fp32 numbers; a row with an infinity
  // takes the smallest, so that its finite values stay finite
  const int e = big > 0.0f ? 13 - max(-113, min(127, ilogbf(big))) : 0;
  const float s = ldexpf(1.0f, e);
  if (threadIdx.x == 0) rs[m] = ldexpf(1.0f, -e);
  _Float16* ar = a + (size_t)m * mats * N;
  for (int n = threadIdx.x * 8; n < N; n += kRowThreads * 8) {
    float dg[8], du[8];
    gradient_group(dH, G, U, row + n, act, mats, dg, du);
    store_group(ar + n, dg, s);
    if (mats == 2) store_group(ar + N + n, du, s);
  }
}

__global__ __launch_bounds__(kRowThreads) void gradient_finish_kernel(
    const float* __restrict__ part, const float* __restrict__ rs, uint16_t* __restrict__ dX,
    int M, int K, int S) {
  typedef uint16_t ushort4v __attribute__((ext_vector_type(4)));
  const size_t mk = (size_t)M * K;
  const size_t i = ((size_t)blockIdx.x * kRowThreads + threadIdx.x) * 4;
  if (i >= mk) return;
  const float r = rs[i / K];
  const float4v v = sum_splits4(part + i, mk, S);
  ushort4v o;
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = float_to_bf16(v[e] * r);
  *reinterpret_cast<ushort4v*>(dX + i) = o;
}

unsigned blocks(size_t n, int per) { return (unsigned)((n + per - 1) / per); }

}  // namespace

hipError_t launch_glu_finish(const float* part, float* h, size_t mn, int S, int act,
                             hipStream_t st) {
  hipLaunchKernelGGL(glu_finish_kernel, dim3(blocks(mn, 64)), dim3(64), 0, st, part, h, mn, S,
                     act);
  return hipGetLastError();
}

hipError_t launch_glu_finish_f16(const float* part, uint16_t* H, uint16_t* G, uint16_t* U,
                                 size_t mn, int S, int act, hipStream_t st) {
  hipLaunchKernelGGL(glu_finish_f16_kernel, dim3(blocks(mn, 4 * kRowThreads)), dim3(kRowThreads),
                     0, st, part, reinterpret_cast<_Float16*>(H), reinterpret_cast<_Float16*>(G),
                     reinterpret_cast<_Float16*>(U), mn, S, act);
  return hipGetLastError();
}

hipError_t launch_lora_shrink(const float* x, const Adapters& ad, float* t, int M, int K,
                              hipStream_t st) {
  hipLaunchKernelGGL(lora_shrink_kernel<float>, dim3(blocks((size_t)M * ad.R, 4)),
                     dim3(kRowThreads), 0, st, x, ad, t, M, K);
  return hipGetLastError();
}

hipError_t launch_lora_shrink_f16(const uint16_t* X, const Adapters& ad, float* t, uint16_t* t16,
                                  float* ts, int M, int K, hipStream_t st) {
  const _Float16* x = reinterpret_cast<const _Float16*>(X);
  if (M <= 64 && !t16) {
    hipLaunchKernelGGL(lora_shrink_kernel<_Float16>, dim3(blocks((size_t)M * ad.R, 4)),
                       dim3(kRowThreads), 0, st, x, ad, t, M, K);
  } else {
    hipLaunchKernelGGL(lora_shrink_tile_kernel, dim3(blocks(M, kShrinkRows)),
                       dim3(kShrinkWaves * kWaveSize), 0, st, x, ad, t,
                       reinterpret_cast<_Float16*>(t16), ts, M, K);
  }
  return hipGetLastError();
}

hipError_t launch_lora_finish(const float* part, const float* t, const Adapters& ad, float* y,
                              int M, int N, int S, hipStream_t st) {
  hipLaunchKernelGGL(lora_finish_kernel<float>, dim3(blocks((size_t)M * N, 64)), dim3(64), 0, st,
                     part, t, ad, y, M, N, S);
  return hipGetLastError();
}

hipError_t launch_lora_finish_f16(const float* part, const float* t, const Adapters& ad,
                                  uint16_t* Y, int M, int N, int S, hipStream_t st) {
  hipLaunchKernelGGL(lora_finish_kernel<_Float16>, dim3(blocks((size_t)M * N, 64)), dim3(64), 0,
                     st, part, t, ad, reinterpret_cast<_Float16*>(Y), M, N, S);
  return hipGetLastError();
}

hipError_t launch_gradient_rows(const uint16_t* dH, const uint16_t* G, const uint16_t* U,
                                uint16_t* a, float* rs, int M, int N, int act, int mats,
                                hipStream_t st) {
  hipLaunchKernelGGL(gradient_rows_kernel, dim3((unsigned)M), dim3(kRowThreads), 0, st, dH, G, U,
                     reinterpret_cast<_Float16*>(a), rs, N, act, mats);
  return hipGetLastError();
}

hipError_t launch_gradient_finish(const float* part, const float* rs, uint16_t* dX, int M, int K,
                                  int S, hipStream_t st) {
  hipLaunchKernelGGL(gradient_finish_kernel, dim3(blocks((size_t)M * K, 4 * kRowThreads)),
                     dim3(kRowThreads), 0, st, part, rs, dX, M, K, S);
  return hipGetLastError();
}

}  // namespace q4
