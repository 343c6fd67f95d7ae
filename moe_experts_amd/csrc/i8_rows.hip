// Row kernels of the 8-bit operators: what stands before and after their products.
//
//   quantize          rows of activations or weights to int8 and one scale each
//   dequantize        and back
//   gradient_rows     dY * sw as the fp16 left operand of the input's gradient
//   gradient_columns  dY * sx, transposed, as that of the weights' gradient
//   finish            results from the split sums of a product
//
// All are bound by memory where they are large: 2048 x 11008 bf16 is quantized in 14.2 us and
// restored in 13.3, 4.8 and 5.1 TB/s of the 67.6 MB that each moves (a large copy reaches 5.1).
// One pass over the data: a row stays in registers between the search for its largest value
// and the rounding, as it stands in memory (converted first, quantizing took 21.3 us, for
// want of waves a CU). Few rows take wider workgroups (8 rows of 11008 fp32: 5.0 -> 3.8 us).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "i8_device.hpp"
#include "i8_internal.hpp"
#include "i8_lost.hpp"

namespace q4 {
namespace {

constexpr int kRowThreads = 256;
constexpr int kFewRows = 256;       // rows by wider workgroups: no more than one a CU
constexpr int kMaxGrid = 1 << 20;  // workgroups; each takes every kMaxGrid-th row after its own

int row_grid(long long n) { return (int)std::min<long long>(n, kMaxGrid); }

// One workgroup a row of at least eight values. V pieces of eight a lane stay in registers
// between the search for the largest and the rounding; LOOP reads longer rows twice. A piece
// that would end behind the row is moved to end with it: some values are then done twice,
// alike. Lanes behind the row repeat its last piece and store nothing.
template <int TYPE, int THREADS, int V, bool LOOP>
__global__ __launch_bounds__(THREADS) void i8_quantize_kernel(
    const typename Val<TYPE>::T* __restrict__ X, int8_t* __restrict__ Q,
    float* __restrict__ scale, int M, int K) {
  __shared__ uint32_t at[THREADS / kWaveSize];
  for (int m = blockIdx.x; m < M; m += gridDim.x) {
    const typename Val<TYPE>::T* xr = X + (size_t)m * K;
    int8_t* qr = Q + (size_t)m * K;
    Piece<TYPE> x[V];
    uint32_t big = 0;
    for (int k0 = 0; k0 < K; k0 += THREADS * 8 * V) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        x[v].load(xr + min(k0 + (v * THREADS + (int)threadIdx.x) * 8, K - 8));
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) big = max(big, magnitude(x[v][e]));
      if (!LOOP) break;
    }
    const RowScale rs = row_scale(workgroup_max<THREADS>(big, at));
    if (threadIdx.x == 0) scale[m] = rs.s;
    for (int k0 = 0; k0 < K; k0 += THREADS * 8 * V) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int k = k0 + (v * THREADS + (int)threadIdx.x) * 8;
        if (LOOP) x[v].load(xr + min(k, K - 8));
        x[v].fresh();
        if (k < K) {
          float f[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = x[v][e];
          uint32_t q[2];
          to_int8<8>(f, rs, q);
          __builtin_memcpy(qr + min(k, K - 8), q, 8);
        }
      }
      if (!LOOP) break;
    }
    if (THREADS > kWaveSize) __syncthreads();  // `at` is read before the next row writes it
  }
}

// Rows of fewer than eight values, one a lane.
template <int TYPE>
__global__ __launch_bounds__(kRowThreads) void i8_quantize_short_kernel(
    const typename Val<TYPE>::T* __restrict__ X, int8_t* __restrict__ Q,
    float* __restrict__ scale, int M, int K) {
  for (long long m = (long long)blockIdx.x * kRowThreads + threadIdx.x; m < M;
       m += (long long)gridDim.x * kRowThreads) {
    float x[8];
    uint32_t big = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[e] = e < K ? Val<TYPE>::get(X[(size_t)m * K + min(e, K - 1)]) : 0.0f;
      big = max(big, magnitude(x[e]));
    }
    const RowScale rs = row_scale(big);
    scale[m] = rs.s;
    uint32_t q[2];
    to_int8<8>(x, rs, q);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < K) Q[(size_t)m * K + e] = (int8_t)(q[e >> 2] >> (8 * (e & 3)));
  }
}

// Eight values a lane, a workgroup a piece of a row of at least eight; the last eight of a row
// as in i8_quantize_kernel.
template <int TYPE, int THREADS>
__global__ __launch_bounds__(THREADS) void i8_dequantize_kernel(
    const int8_t* __restrict__ Q, const float* __restrict__ scale,
    typename Val<TYPE>::T* __restrict__ X, int M, int K, int pieces) {
  for (long long i = blockIdx.x; i < (long long)M * pieces; i += gridDim.x) {
    const int m = (int)(i / pieces);
    const int k = ((int)(i % pieces) * THREADS + (int)threadIdx.x) * 8;
    if (k >= K) continue;
    const size_t at = (size_t)m * K + min(k, K - 8);
    const float s = scale[m];
    int8_t q[8];
    __builtin_memcpy(q, Q + at, 8);
    typename Val<TYPE>::T v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = Val<TYPE>::put((float)q[e] * s);
    __builtin_memcpy(X + at, v, sizeof(v));
  }
}

// Rows of fewer than eight values, a value a lane.
template <int TYPE>
__global__ __launch_bounds__(kRowThreads) void i8_dequantize_short_kernel(
    const int8_t* __restrict__ Q, const float* __restrict__ scale,
    typename Val<TYPE>::T* __restrict__ X, long long n, int K) {
  for (long long i = (long long)blockIdx.x * kRowThreads + threadIdx.x; i < n;
       i += (long long)gridDim.x * kRowThreads)
    X[i] = Val<TYPE>::put((float)Q[i] * scale[i / K]);
}

// One workgroup a row of dY; N and ld are multiples of 8.
template <int THREADS, int V, bool LOOP>
__global__ __launch_bounds__(THREADS) void i8_gradient_rows_kernel(
    const uint16_t* __restrict__ dY, const float* __restrict__ sw, LeftOperand l, int M, int N) {
  __shared__ uint32_t at[THREADS / kWaveSize], units;
  const int ld = l.ld;
  for (int m = blockIdx.x; m < M; m += gridDim.x) {
    if (threadIdx.x == 0) units = 0;
    const uint16_t* yr = dY + (size_t)m * N;
    uint16_t* ar = l.a + (size_t)m * ld;
    float x[V][8];
    // products of the pieces from n0 on, zeros behind the row
    auto load = [&](int n0) {
      Piece<Q4_TYPE_BF16> y[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int n = min(n0 + (v * THREADS + (int)threadIdx.x) * 8, N - 8);
        y[v].load(yr + n);
        __builtin_memcpy(x[v], sw + n, 32);
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const bool in = n0 + (v * THREADS + (int)threadIdx.x) * 8 < N;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[v][e] = in ? y[v][e] * x[v][e] : 0.0f;
      }
    };
    uint32_t big = 0, least = kNoLeast;
    for (int n0 = 0; n0 < N; n0 += THREADS * 8 * V) {
      load(n0);
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          big = max(big, magnitude(x[v][e]));
          least = least_of(least, x[v][e]);
        }
      if (!LOOP) break;
    }
    const PowerOfTwo p = to_fp16_range(workgroup_max<THREADS>(big, at));
    if (threadIdx.x == 0) l.rs[m] = p.down;
    const bool losing = may_lose(least, p.up);
    for (int n0 = 0; n0 < ld; n0 += THREADS * 8 * V) {
      if (LOOP) load(n0);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int n = n0 + (v * THREADS + (int)threadIdx.x) * 8;
        if (n >= ld) continue;
        half8 h;
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = (_Float16)(x[v][e] * p.up);
        *reinterpret_cast<half8*>(ar + n) = h;
        if (losing) {
          float gone = 0.0f;
#pragma unroll
          for (int e = 0; e < 8; ++e) gone += fabsf(lost16(x[v][e] * p.up));
          add_lost(&units, gone);
        }
      }
      if (!LOOP) break;
    }
    lds_only_barrier();
    const uint32_t sum = units;
    if (threadIdx.x == 0) l.lost[m] = sum;
    for (int n0 = 0; sum != 0 && n0 < ld; n0 += THREADS * 8 * V) {
      if (LOOP) load(n0);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int n = n0 + (v * THREADS + (int)threadIdx.x) * 8;
        if (n >= ld) continue;
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w[e] = lost_bf16(x[v][2 * e] * p.up) | lost_bf16(x[v][2 * e + 1] * p.up) << 16;
        *reinterpret_cast<uint4*>(l.a2 + (size_t)m * ld + n) = make_uint4(w[0], w[1], w[2], w[3]);
      }
      if (!LOOP) break;
    }
    lds_only_barrier();  // `units` is read before the next row clears it
  }
}

// ---------------------------------------------------------------------------
// dY * sx by columns, up to kOnceRows rows: one workgroup holds eight columns of all rows in
// registers, so that dY is read once for the search and the rounding. A lane has P pairs of
// neighbouring rows; a pair's values of a column are one dword of the result, and 64 lanes
// store 256 bytes of a column together. The 16 bytes of a row share their line with those of
// seven other workgroups, which run on the same XCD. Against the two kernels below, us a call of the
// gradient on the GPU: 777 rows of 5120 x 1536 27.0 and 33.0, 2048 of 4096 x 4096 81.3 and 86.1, 8192
// of 4096 x 4096 306 and 304; but 2048 of 4096 x 11008, whose dY comes from memory, 222 and 215, of
// 1024 x 11008 79.7 and 78.8: hence kOnceCols.
// ---------------------------------------------------------------------------
constexpr int kOnceRows = 8192, kOnceCols = 4096;
bool columns_once(int M, int N) { return M <= kOnceRows && N <= kOnceCols; }

template <int THREADS, int P>
__global__ __launch_bounds__(THREADS) void i8_gradient_columns_once_kernel(
    const uint16_t* __restrict__ dY, const float* __restrict__ sx, LeftOperand l, int M, int N) {
  const int ld = l.ld;
  constexpr int kWaves = THREADS / kWaveSize;
  __shared__ uint32_t at[kWaves][8], units[8];
  __shared__ float factor[8];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int n = xcd_logical_tile(blockIdx.x, gridDim.x) * 8;
  Piece<Q4_TYPE_BF16> v[P][2];
  float s[P][2];
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int m = 2 * (p * THREADS + t) + h;
      v[p][h].load(dY + (size_t)min(m, M - 1) * N + n);
      s[p][h] = sx[min(m, M - 1)];
    }
  // rows past the last are zeros, whatever the one that was read in their place holds
  auto value = [&](int p, int h, int e) {
    return 2 * (p * THREADS + t) + h < M ? v[p][h][e] * s[p][h] : 0.0f;
  };
  uint32_t big[8] = {}, least[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) least[e] = kNoLeast;
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float f = value(p, h, e);
        big[e] = max(big[e], magnitude(f));
        least[e] = least_of(least[e], f);
      }
  const int e = wave_max_of_eight<1>(big);
  if (lane < 8) at[wave][e] = big[0];
  __syncthreads();
  if (t < kWaveSize) {  // wave 0: lane l column l % 8 of every eighth wave
    uint32_t b = 0;
#pragma unroll
    for (int w = 0; w < kWaves; w += 8)
      if (w + (lane >> 3) < kWaves) b = max(b, at[w + (lane >> 3)][lane & 7]);
#pragma unroll
    for (int o = 8; o < kWaveSize; o <<= 1) b = max(b, (uint32_t)__shfl_xor((int)b, o));
    const PowerOfTwo f = to_fp16_range(b);
    if (lane < 8) {
      factor[lane] = f.up;
      l.rs[n + lane] = f.down;
      units[lane] = 0;
    }
  }
  __syncthreads();
  float low = 1.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float up = factor[e];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int m = 2 * (p * THREADS + t);  // ld is even
      if (m < ld)
        *reinterpret_cast<half2v*>(l.a + (size_t)(n + e) * ld + m) =
            half2v{(_Float16)(value(p, 0, e) * up), (_Float16)(value(p, 1, e) * up)};
    }
    low = fminf(low, scaled_least(least[e], up));
  }
  if (low < kLeast16)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float gone = 0.0f;
#pragma unroll
      for (int p = 0; p < P; ++p)
        gone += fabsf(lost16(value(p, 0, e) * factor[e])) + fabsf(lost16(value(p, 1, e) * factor[e]));
      add_lost(&units[e], gone);
    }
  lds_only_barrier();
  const uint32_t sum = units[lane & 7];
  if (t < 8) l.lost[n + t] = sum;
  if (!__any(sum != 0)) return;  // the same in all waves
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if (units[e] == 0) continue;  // uniform
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int m = 2 * (p * THREADS + t);
      if (m < ld)
        *reinterpret_cast<uint32_t*>(l.a2 + (size_t)(n + e) * ld + m) =
            lost_bf16(value(p, 0, e) * factor[e]) | lost_bf16(value(p, 1, e) * factor[e]) << 16;
    }
  }
}

// Largest and least |dY * sx| (i8_lost.hpp) of 64 columns in a chunk of the rows. Every workgroup of
// the second kernel reads all chunks' values of its columns, so there are at most kMaxChunks.
constexpr int kCols = 64, kColLanes = kCols / 8, kRowLanes = kRowThreads / kColLanes;
constexpr int kChunkRows = 256, kMaxChunks = 64;

int max_rows(int M) {  // of a chunk
  const int least = (M + kMaxChunks - 1) / kMaxChunks;
  return std::max(kChunkRows, (least + kRowLanes - 1) / kRowLanes * kRowLanes);
}

__global__ __launch_bounds__(kRowThreads) void i8_column_max_kernel(
    const uint16_t* __restrict__ dY, const float* __restrict__ sx, uint32_t* __restrict__ big,
    uint32_t* __restrict__ least, uint32_t* __restrict__ lost, int M, int N, int tiles_n,
    int chunk_rows) {
  __shared__ uint32_t at[2][kRowLanes][kCols];
  const int c8 = (int)threadIdx.x % kColLanes, r = (int)threadIdx.x / kColLanes;
  const int n = ((int)blockIdx.x % tiles_n) * kCols + c8 * 8;
  const int chunk = (int)blockIdx.x / tiles_n;
  uint32_t b[8] = {}, s8[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) s8[e] = kNoLeast;
  if (n < N) {
    const int m1 = (int)min((long long)M, (long long)(chunk + 1) * chunk_rows);
#pragma unroll 8
    for (int m = chunk * chunk_rows + r; m < m1; m += kRowLanes) {
      uint16_t v[8];
      __builtin_memcpy(v, __builtin_assume_aligned(dY + (size_t)m * N + n, 16), 16);
      const float s = sx[m];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float f = Val<Q4_TYPE_BF16>::get(v[e]) * s;
        b[e] = max(b[e], magnitude(f));
        s8[e] = least_of(s8[e], f);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    at[0][r][c8 * 8 + e] = b[e];
    at[1][r][c8 * 8 + e] = s8[e];
  }
  __syncthreads();
  if (threadIdx.x < kCols) {
    uint32_t v = 0, s = kNoLeast;
#pragma unroll
    for (int i = 0; i < kRowLanes; ++i) {
      v = max(v, at[0][i][threadIdx.x]);
      s = min(s, at[1][i][threadIdx.x]);
    }
    const int col = ((int)blockIdx.x % tiles_n) * kCols + (int)threadIdx.x;
    if (col < N) {
      big[(size_t)chunk * N + col] = v;
      least[(size_t)chunk * N + col] = s;
      if (chunk == 0) lost[col] = 0;  // for the second kernel
    }
  }
}

// 64 columns by kChunkRows rows of dY, all read at once, then transposed through LDS 128 rows at
// a time: two neighbouring rows of a column are a dword, and 64 lanes store 256 bytes of a
// column.
__global__ __launch_bounds__(kRowThreads) void i8_gradient_columns_kernel(
    const uint16_t* __restrict__ dY, const float* __restrict__ sx,
    const uint32_t* __restrict__ big, const uint32_t* __restrict__ least, LeftOperand l, int M,
    int N, int tiles_n, int chunks) {
  const int ld = l.ld;
  constexpr int kPairs = kChunkRows / 2 / kRowLanes;  // of a lane
  constexpr int kPitch = 64 + 1;  // dwords of a column: eight columns on are eight banks on
  __shared__ uint32_t tile[kCols * kPitch];
  __shared__ float up[kCols];
  __shared__ uint32_t units[kCols];
  __shared__ uint64_t losing;  // a bit a column
  const int n0 = ((int)blockIdx.x % tiles_n) * kCols;
  const int m0 = (int)blockIdx.x / tiles_n * kChunkRows;
  const int c8 = (int)threadIdx.x % kColLanes, r = (int)threadIdx.x / kColLanes;
  const int n = min(n0 + c8 * 8, N - 8);  // columns past the last are not stored
  Piece<Q4_TYPE_BF16> v[kPairs][2];
  float s[kPairs][2];
#pragma unroll
  for (int p = 0; p < kPairs; ++p)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int m = min(m0 + 2 * (p * kRowLanes + r) + h, M - 1);
      v[p][h].load(dY + (size_t)m * N + n);
      s[p][h] = sx[m];
    }
  if (threadIdx.x < kCols) {
    const int col = n0 + (int)threadIdx.x;
    uint32_t b = 0, low = kNoLeast;
    if (col < N)
      for (int c = 0; c < chunks; ++c) {
        b = max(b, big[(size_t)c * N + col]);
        low = min(low, least[(size_t)c * N + col]);
      }
    const PowerOfTwo f = to_fp16_range(b);
    up[threadIdx.x] = f.up;
    units[threadIdx.x] = 0;
    if (col < N && m0 == 0) l.rs[col] = f.down;
    const uint64_t some = __ballot(may_lose(low, f.up));
    if (threadIdx.x == 0) losing = some;
  }
  __syncthreads();
  float u[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) u[e] = up[c8 * 8 + e];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int p = 0; p < kPairs; p += 2) {
    const int mt = m0 + 2 * p * kRowLanes;  // first of the 128 rows
    if (mt >= ld) break;                    // uniform
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        half2v h;
#pragma unroll
        for (int j = 0; j < 2; ++j)
          h[j] = m0 + 2 * ((p + i) * kRowLanes + r) + j < M
                     ? (_Float16)(v[p + i][j][e] * s[p + i][j] * u[e])
                     : (_Float16)0.0f;
        tile[(c8 * 8 + e) * kPitch + i * kRowLanes + r] = __builtin_bit_cast(uint32_t, h);
      }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kCols; i += kRowThreads / kWaveSize) {
      const int col = i + wave, m = mt + 2 * lane;  // ld is even
      if (n0 + col < N && m < ld)
        *reinterpret_cast<uint32_t*>(l.a + (size_t)(n0 + col) * ld + m) = tile[col * kPitch + lane];
    }
    __syncthreads();
  }
  const uint64_t some = losing;
  if (some == 0) return;  // uniform
  // Columns that have, in this chunk or another, something to lose: all chunks write what theirs do,
  // a lane one row, four columns at a time. (By LDS as above 11008 columns, of which 22 lose a
  // value, took 27 us instead of 18.)
  static_assert(kChunkRows == kRowThreads, "a row a lane");
  const int m = m0 + (int)threadIdx.x;
  const float f = m < M ? sx[m] : 0.0f;
#pragma unroll 1
  for (uint64_t left = some; left != 0;) {
    int col[4];
    float x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // the last again where fewer are left
      col[i] = left != 0 || i == 0 ? __builtin_ctzll(left) : col[i ? i - 1 : 0];
      left &= left - 1;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[i] = Val<Q4_TYPE_BF16>::get(dY[(size_t)min(m, M - 1) * N + n0 + col[i]]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i > 0 && col[i] == col[i - 1]) break;  // uniform
      const float v = m < M ? x[i] * f * up[col[i]] : 0.0f;
      if (m < ld) l.a2[(size_t)(n0 + col[i]) * ld + m] = (uint16_t)lost_bf16(v);
      float gone = fabsf(lost16(v));
      if (!__any(gone > 0.0f)) continue;
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) gone += __shfl_xor(gone, o);
      if (lane == 0) add_lost(&units[col[i]], gone);
    }
  }
  lds_only_barrier();
  if (threadIdx.x < kCols && units[threadIdx.x] != 0)  // of a column before the last
    atomicAdd(&l.lost[n0 + (int)threadIdx.x], units[threadIdx.x]);
}

// ---------------------------------------------------------------------------
// Sums of splits, in split order, four results a lane. Eight loads at a time are issued
// before the first addition; those past the last split repeat it and are not added.
// ---------------------------------------------------------------------------
template <class V>
__device__ __forceinline__ V sum_splits(const V* __restrict__ p, size_t stride, int S) {
  V sum{};
  for (int s0 = 0; s0 < S; s0 += 8) {
    V t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = p[(size_t)min(s0 + i, S - 1) * stride];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (s0 + i < S) sum += t[i];
  }
  return sum;
}

template <int TYPE>
__global__ __launch_bounds__(kRowThreads) void i8_finish_kernel(
    const int32_t* __restrict__ part, const float* __restrict__ sx, const float* __restrict__ sw,
    typename Val<TYPE>::T* __restrict__ Y, size_t mn, int N, int S) {
  const size_t i = ((size_t)blockIdx.x * kRowThreads + threadIdx.x) * 4;
  if (i >= mn) return;
  const int m = (int)(i / N), n = (int)(i - (size_t)m * N);
  const int4v v = sum_splits(reinterpret_cast<const int4v*>(part + i), mn / 4, S);
  const float s = sx[m];
  typename Val<TYPE>::T y[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = Val<TYPE>::put((float)v[e] * s * sw[n + e]);
  __builtin_memcpy(__builtin_assume_aligned(Y + i, sizeof(y)), y, sizeof(y));
}

__global__ __launch_bounds__(kRowThreads) void i8_gradient_finish_kernel(
    const float* __restrict__ part, const float* __restrict__ rs, uint16_t* __restrict__ out,
    size_t mn, int cols, int S) {
  const size_t i = ((size_t)blockIdx.x * kRowThreads + threadIdx.x) * 4;
  if (i >= mn) return;
  const float4v v = sum_splits(reinterpret_cast<const float4v*>(part + i), mn / 4, S);
  const float s = rs ? rs[i / cols] : 1.0f;
  uint16_t y[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = (uint16_t)i8_to_bf16(v[e] * s);
  __builtin_memcpy(__builtin_assume_aligned(out + i, 8), y, 8);
}

template <int TYPE, int THREADS, int V, bool LOOP>
void quantize(const void* X, int8_t* Q, float* scale, int M, int K, hipStream_t st) {
  hipLaunchKernelGGL((i8_quantize_kernel<TYPE, THREADS, V, LOOP>), dim3(row_grid(M)),
                     dim3(THREADS), 0, st, static_cast<const typename Val<TYPE>::T*>(X), Q, scale,
                     M, K);
}

template <int THREADS, int V, bool LOOP>
void gradient_rows(const uint16_t* dY, const float* sw, const LeftOperand& l, int M, int N,
                   hipStream_t st) {
  hipLaunchKernelGGL((i8_gradient_rows_kernel<THREADS, V, LOOP>), dim3(row_grid(M)),
                     dim3(THREADS), 0, st, dY, sw, l, M, N);
}

// The compiled forms of a kernel: threads, pieces of eight values a lane, passes over the data.
template <int THREADS, int PIECES, int PASSES>
struct Form {
  static constexpr int kThreads = THREADS, kPieces = PIECES, kPasses = PASSES;
};
template <class... F>
struct Forms {};
typedef Forms<Form<64, 1, 1>, Form<256, 1, 1>, Form<256, 2, 1>, Form<256, 4, 1>, Form<256, 6, 1>,
              Form<256, 8, 1>, Form<256, 4, 2>>
    RowForms;
typedef Forms<Form<64, 1, 1>, Form<256, 1, 1>, Form<256, 2, 1>, Form<256, 4, 1>, Form<256, 6, 1>,
              Form<256, 8, 1>, Form<256, 4, 2>, Form<1024, 1, 1>, Form<1024, 2, 1>>
    QuantizeForms;
typedef Forms<Form<64, 2, 1>, Form<256, 2, 1>, Form<512, 2, 1>, Form<1024, 2, 1>, Form<1024, 4, 1>,
              Form<1024, 8, 1>>
    ColumnForms;

// Calls `go` with the form that a plan names; false if there is none.
template <class Go, class... F>
bool by_form(const I8RowsPlan& p, Forms<F...>, Go&& go) {
  auto one = [&](auto form) {
    using T = decltype(form);
    if (p.threads != T::kThreads || p.pieces != T::kPieces || p.passes != T::kPasses) return false;
    go(form);
    return true;
  };
  return (one(F{}) || ...);
}

}  // namespace

// Rows of fewer than eight values have a kernel of their own (pieces 0).
I8RowsPlan plan_i8_quantize(int M, int K) {
  if (K < 8) return {kRowThreads, 0, 1};
  if (K <= 512) return {64, 1, 1};
  if (K <= 2048) return {256, 1, 1};
  if (M <= kFewRows && K <= 8192) return {1024, 1, 1};
  if (M <= kFewRows && K <= 16384) return {1024, 2, 1};
  if (K <= 4096) return {256, 2, 1};
  if (K <= 8192) return {256, 4, 1};
  if (K <= 12288) return {256, 6, 1};
  if (K <= 16384) return {256, 8, 1};
  return {256, 4, 2};
}

hipError_t launch_i8_quantize(const void* X, int type, int8_t* Q, float* scale, int M, int K,
                              hipStream_t st) {
  const I8RowsPlan p = plan_i8_quantize(M, K);
  bool found = false;
  i8_by_type(type, [&](auto t) {
    constexpr int TYPE = decltype(t)::value;
    if (p.pieces == 0) {
      found = true;
      hipLaunchKernelGGL((i8_quantize_short_kernel<TYPE>),
                         dim3(row_grid(((long long)M + kRowThreads - 1) / kRowThreads)),
                         dim3(kRowThreads), 0, st, static_cast<const typename Val<TYPE>::T*>(X), Q,
                         scale, M, K);
      return;
    }
    found = by_form(p, QuantizeForms{}, [&](auto form) {
      using F = decltype(form);
      quantize<TYPE, F::kThreads, F::kPieces, F::kPasses == 2>(X, Q, scale, M, K, st);
    });
  });
  return found ? hipGetLastError() : hipErrorInvalidValue;
}

hipError_t launch_i8_dequantize(const int8_t* Q, const float* scale, void* X, int type, int M,
                                int K, hipStream_t st) {
  i8_by_type(type, [&](auto t) {
    constexpr int TYPE = decltype(t)::value;
    typedef typename Val<TYPE>::T T;
    if (K < 8) {
      const long long n = (long long)M * K;
      hipLaunchKernelGGL((i8_dequantize_short_kernel<TYPE>),
                         dim3(row_grid((n + kRowThreads - 1) / kRowThreads)), dim3(kRowThreads), 0,
                         st, Q, scale, static_cast<T*>(X), n, K);
    } else if (K <= 512) {
      hipLaunchKernelGGL((i8_dequantize_kernel<TYPE, 64>), dim3(row_grid(M)), dim3(64), 0, st, Q,
                         scale, static_cast<T*>(X), M, K, 1);
    } else {
      const int pieces = (K - 1) / (kRowThreads * 8) + 1;
      hipLaunchKernelGGL((i8_dequantize_kernel<TYPE, kRowThreads>),
                         dim3(row_grid((long long)M * pieces)), dim3(kRowThreads), 0, st, Q, scale,
                         static_cast<T*>(X), M, K, pieces);
    }
  });
  return hipGetLastError();
}

I8RowsPlan plan_i8_gradient_rows(int ld) {
  if (ld <= 512) return {64, 1, 1};
  if (ld <= 2048) return {256, 1, 1};
  if (ld <= 4096) return {256, 2, 1};
  if (ld <= 8192) return {256, 4, 1};
  if (ld <= 12288) return {256, 6, 1};
  if (ld <= 16384) return {256, 8, 1};
  return {256, 4, 2};
}

hipError_t launch_i8_gradient_rows(const uint16_t* dY, const float* sw, const LeftOperand& l, int M,
                                   int N, hipStream_t st) {
  const bool found = by_form(plan_i8_gradient_rows(l.ld), RowForms{}, [&](auto form) {
    using F = decltype(form);
    gradient_rows<F::kThreads, F::kPieces, F::kPasses == 2>(dY, sw, l, M, N, st);
  });
  return found ? hipGetLastError() : hipErrorInvalidValue;
}

// Pieces: of a lane, in pairs of rows where one kernel does it all.
I8RowsPlan plan_i8_gradient_columns(int M, int N, int ld) {
  if (!columns_once(M, N)) return {kRowThreads, kChunkRows / kRowLanes, 2};
  if (ld <= 128) return {64, 2, 1};
  if (ld <= 512) return {256, 2, 1};
  if (ld <= 1024) return {512, 2, 1};
  if (ld <= 2048) return {1024, 2, 1};
  if (ld <= 4096) return {1024, 4, 1};
  return {1024, 8, 1};
}

int i8_max_chunks(int M, int N) {
  return columns_once(M, N) ? 0 : (M + max_rows(M) - 1) / max_rows(M);
}

hipError_t launch_i8_gradient_columns(const uint16_t* dY, const float* sx, const LeftOperand& l,
                                      uint32_t* scratch, int M, int N, hipStream_t st) {
  const I8RowsPlan p = plan_i8_gradient_columns(M, N, l.ld);
  if (p.passes == 1) {
    const bool found = by_form(p, ColumnForms{}, [&](auto form) {
      using F = decltype(form);
      hipLaunchKernelGGL((i8_gradient_columns_once_kernel<F::kThreads, F::kPieces / 2>),
                         dim3((unsigned)(N / 8)), dim3(F::kThreads), 0, st, dY, sx, l, M, N);
    });
    return found ? hipGetLastError() : hipErrorInvalidValue;
  }
  const int tiles_n = (N + kCols - 1) / kCols, maxima = i8_max_chunks(M, N);
  const long long grid = (long long)tiles_n * ((M + kChunkRows - 1) / kChunkRows);
  if (grid > 0xffffffLL) return hipErrorInvalidValue;  // below 2^32 lanes
  uint32_t* big = scratch;
  uint32_t* least = scratch + (size_t)maxima * N;
  hipLaunchKernelGGL(i8_column_max_kernel, dim3((unsigned)(tiles_n * maxima)), dim3(kRowThreads), 0,
                     st, dY, sx, big, least, l.lost, M, N, tiles_n, max_rows(M));
  hipLaunchKernelGGL(i8_gradient_columns_kernel, dim3((unsigned)grid), dim3(kRowThreads), 0, st,
                     dY, sx, big, least, l, M, N, tiles_n, maxima);
  return hipGetLastError();
}

hipError_t launch_i8_finish(const int32_t* part, const float* sx, const float* sw, void* Y,
                            int type, int M, int N, int S, hipStream_t st) {
  const size_t mn = (size_t)M * N;
  const unsigned grid = (unsigned)((mn / 4 + kRowThreads - 1) / kRowThreads);
  i8_by_type(type, [&](auto t) {
    constexpr int TYPE = decltype(t)::value;
    hipLaunchKernelGGL((i8_finish_kernel<TYPE>), dim3(grid), dim3(kRowThreads), 0, st, part, sx, sw,
                       static_cast<typename Val<TYPE>::T*>(Y), mn, N, S);
  });
  return hipGetLastError();
}

hipError_t launch_i8_gradient_finish(const float* part, const float* rs, uint16_t* out, int rows,
                                     int cols, int S, hipStream_t st) {
  const size_t mn = (size_t)rows * cols;
  const unsigned grid = (unsigned)((mn / 4 + kRowThreads - 1) / kRowThreads);
  hipLaunchKernelGGL(i8_gradient_finish_kernel, dim3(grid), dim3(kRowThreads), 0, st, part, rs, out,
                     mn, cols, S);
  return hipGetLastError();
}

}  // namespace q4
