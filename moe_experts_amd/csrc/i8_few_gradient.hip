// Gradients of the 8-bit product with few rows in the result, or little work, in one kernel:
//   weights (an adapter's rank of output channels)
//     dW[n][k] = sum_m (dY[m][n] * sx[m]) * X[m][k]
//   input
//     dX[m][k] = sum_n (dY[m][n] * sw[n]) * W[n][k]
// or C[i][k] = sum_c A[i][c] * B[c][k]. A workgroup makes 16 rows and 64 columns of C. Of B its
// columns' rows are on their way into LDS while it makes its rows of A: dY times the scales,
// scaled row by row of C and rounded to fp16 as for the tiles, in LDS with c contiguous. Its
// waves then share out the rows of B: each multiplies steps of 32 by v_mfma_f32_16x16x32_f16,
// copied memory -> LDS several steps ahead into a part of its own, and their sums meet in LDS,
// in the order of the waves. Where a result may rest on what the rounding of A has lost, the
// workgroup goes over the contraction a second time with that in A's place (i8_lost.hpp).
//
// A contraction of up to 2048 (4096 with up to 8 rows) fits a workgroup of eight waves; a longer
// one (of the weights' gradient) is split over workgroups of four waves and half as much, two
// of which fit a CU. Each split scales by the power of two of its own part and takes it back
// (exact), so splits are sums of their own, added in their order by a second kernel.
//
// What bounds it: rank 16 of 1999 rows of 11008 10.1 us, of which B takes 4.4 at a large copy's
// rate; the rest is the start, dY's way from memory and its 32768 values' conversion (a
// microsecond on a CU's four units, and 0.35 for the search for what it loses, i8_lost.hpp), which
// the copies in flight only hide as far as they fit LDS. By a transposing kernel and the tiles:
// 16.6. Rank 16 of 8192 rows of 4096 14.7 us (tiles 21.5), of 11008 31.5 (31.2), of 4096 rows of
// 4096 11.2 (16.6), of a row 5.9 (7.2). Four waves and eight took the same at rank 16 of 8192 rows
// of 4096 (12.9 and 12.7, without the search), four less at 11008 (27.8 and 29.2) and at 4096 rows
// (9.5 and 10.7). Past 64 splits the tiles take over.
//
// More than 16 rows, and the input's gradient, take it where no splits are needed, the former up
// to kGroups workgroups, one a CU (eight waves' LDS leaves no room for two, and four waves hold
// half the contraction): it saves the launch that writes A, 2.7 us from a program that launches
// call by call. On the GPU alone, us, here and by tiles: weights of 64 x 512 over 64 rows 5.8 and
// 7.3, 256 x 1024 over 1000 8.2 and 11.9, 64 x 4096 over 2048 (256 workgroups) 12.9 and 17.4; input,
// 4 rows of 1536 x 5120 8.8 and 11.5, 64 of 2048 x 4096 (256) 11.2 and 13.4, 128 of 128 x 256 6.3 and
// 6.5, one of 4096 x 4096 12.9 and 11.6. With more workgroups than CUs: weights of 24 x 11008 over
// 1999 (344) 19.4 and 16.9, 32 x 11008 20.0 and 17.7, 72 x 4096 over 2000 (320) 21.1 and 17.3,
// 512 x 1024 over 1000 (512) 14.8 and 12.2; input, 80 rows of 2048 x 4096 (320) 17.8 and 13.7. The
// input's split: 16 of 8192 x 16384 39.5 and 31.4, without the search.
#include <algorithm>

#include "i8_device.hpp"
#include "i8_internal.hpp"
#include "i8_lost.hpp"
#include "i8_tile.hpp"

namespace q4 {
namespace {

constexpr int kCols = 64;          // of B, a workgroup
constexpr int kStepRows = 32;      // of B, a step of a wave
constexpr int kStepCopy = kStepRows * kCols;
constexpr int NS = 5;              // steps of a wave in LDS
constexpr int kWaveValues = 4096;  // of A in LDS, a wave
constexpr int kGroups = 256;       // workgroups, where the result has more than 16 rows

struct FewArgs {
  const uint16_t* dY;  // [depth][rows], or of the input's gradient [rows][depth]
  const float* scale;  // [depth]
  const int8_t* B;     // [depth][cols]
  uint16_t* out;       // [rows][cols]
  float* part;         // fp32 [S][rows][cols]
  int rows, depth, cols, tiles, groups, S, chunk;
};
// The rows of the result that a workgroup makes: `count` from `first` on.
struct Group {
  int first, count;
};

// Where the 16-byte chunk c of a step's row k stands: c ^ swz_step(k). The rows that 32 lanes
// read at once, 16 of one chunk, meet no bank twice.
__device__ __forceinline__ int swz_step(int k) { return 2 * ((k >> 2) & 1) + ((k >> 3) & 1); }

// A workgroup's share of dY, 64 values a lane, [p][e], in registers. N rows of A, 8 or 16.
// Parts past the end are the last times zero: zeros, or a NaN in a row of A that holds an
// infinity or a NaN there and so has no finite result.
//
// For the weights dY is transposed on its way: value p, e of a lane is column 8 * half + e of its
// row 2 * (p / 2 * kLanes + at) + p % 2; pairs of rows are a dword of A.
template <int N, int THREADS>
struct Transposed {
  static constexpr int kPieces = N / 8, kLanes = THREADS / kPieces, kPer = 2 * kLanes;
  Piece<Q4_TYPE_BF16> v[8];
  float s[8];
  int half, at;
  __device__ __forceinline__ void load(const FewArgs& g, const Group& r, int c0, int left) {
    half = threadIdx.x % kPieces;
    at = threadIdx.x / kPieces;
    const uint16_t* y = g.dY + r.first + min(8 * half, r.count - 8);  // rows is a multiple of 8
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      const int c = c0 + min(p / 2 * kPer + 2 * at + p % 2, left - 1);
      v[p].load(y + (size_t)c * g.rows);
      s[p] = g.scale[c];
    }
  }
  // whether any lane's value p is of use; uniform
  static __device__ __forceinline__ bool used(int p, const Group&, int left) {
    return p / 2 * kPer < left;
  }
  __device__ __forceinline__ void multiply(float (&x)[8], int p, int left) const {
    const float f = p / 2 * kPer + 2 * at + p % 2 < left ? s[p] : 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = v[p][e] * f;
  }
  // the largest of every row of A in this wave, the least of a lane's values of each (i8_lost.hpp)
  uint32_t least[8];
  __device__ __forceinline__ void largest(const float (&x)[8][8], const Group& r, int left,
                                          uint32_t* big) {
    float m[8] = {};
#pragma unroll
    for (int e = 0; e < 8; ++e) least[e] = kNoLeast;
#pragma unroll
    for (int p = 0; p < 8; p += 2)
      if (used(p, r, left))
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          m[e] = fmaxf(fmaxf(m[e], fabsf(x[p][e])), fabsf(x[p + 1][e]));
          least[e] = least_of(least_of(least[e], x[p][e]), x[p + 1][e]);
        }
    uint32_t b[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) b[e] = magnitude(m[e]);
    const int e = wave_max_of_eight<kPieces>(b);
    if ((threadIdx.x & 63) < N) big[8 * half + e] = b[0];
  }
  // the waves that hold values of row i
  static __device__ __forceinline__ int first_wave(int) { return 0; }
  static constexpr int kWavesOfRow = THREADS / kWaveSize;
  __device__ __forceinline__ void store(const float (&x)[8][8], uint8_t* a, int pitch,
                                        const float* up, uint32_t* lost, const Group& r,
                                        int left) const {
#pragma unroll
    for (int p = 0; p < 8; p += 2)
      if (used(p, r, left))  // and so all of the last step
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float f = up[8 * half + e];
          *reinterpret_cast<half2v*>(a + (8 * half + e) * pitch + p * kPer + 4 * at) =
              half2v{(_Float16)(x[p][e] * f), (_Float16)(x[p + 1][e] * f)};
        }
    float low = 1.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) low = fminf(low, scaled_least(least[e], up[8 * half + e]));
    if (low >= kLeast16) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float f = up[8 * half + e];
      float gone = 0.0f;
#pragma unroll
      for (int p = 0; p < 8; p += 2)
        if (used(p, r, left)) gone += fabsf(lost16(x[p][e] * f)) + fabsf(lost16(x[p + 1][e] * f));
      add_lost(&lost[8 * half + e], gone);
    }
  }
  // what store() has lost, as bf16 numbers
  __device__ __forceinline__ void store_lost(const float (&x)[8][8], uint8_t* a, int pitch,
                                             const float* up, const Group& r, int left) const {
#pragma unroll
    for (int p = 0; p < 8; p += 2)
      if (used(p, r, left))
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float f = up[8 * half + e];
          *reinterpret_cast<uint32_t*>(a + (8 * half + e) * pitch + p * kPer + 4 * at) =
              lost_bf16(x[p][e] * f) | lost_bf16(x[p + 1][e] * f) << 16;
        }
  }
};

// For the input dY stands as A does: value p, e of a lane is column 8 * at + e of row
// p * kPieces + part. Rows past the last repeat it and are not kept.
template <int N, int THREADS>
struct Straight {
  static constexpr int kPieces = N / 8, kLanes = THREADS / kPieces;
  Piece<Q4_TYPE_BF16> v[8];
  float s[8];
  int part, at;
  __device__ __forceinline__ void load(const FewArgs& g, const Group& r, int c0, int left) {
    part = __builtin_amdgcn_readfirstlane(threadIdx.x / kLanes);
    at = threadIdx.x % kLanes;
    const int c = c0 + min(8 * at, left - 8);  // depth and left are multiples of 8
#pragma unroll
    for (int p = 0; p < 8; ++p)
      v[p].load(g.dY + (size_t)(r.first + min(p * kPieces + part, r.count - 1)) * g.depth + c);
    __builtin_memcpy(s, g.scale + c, sizeof(s));
  }
  static __device__ __forceinline__ constexpr bool used(int, const Group&, int) { return true; }
  __device__ __forceinline__ void multiply(float (&x)[8], int p, int left) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = v[p][e] * (8 * at < left ? s[e] : 0.0f);
  }
  uint32_t least[8];
  __device__ __forceinline__ void largest(const float (&x)[8][8], const Group& r, int left,
                                          uint32_t* big) {
    uint32_t b[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      float m = 0.0f;
      least[p] = kNoLeast;
      if (used(p, r, left))
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          m = fmaxf(m, fabsf(x[p][e]));
          least[p] = least_of(least[p], x[p][e]);
        }
      b[p] = magnitude(m);
    }
    const int p = wave_max_of_eight<1>(b);
    if ((threadIdx.x & 63) < 8) big[p * kPieces + part] = b[0];
  }
  static constexpr int kWavesOfRow = kLanes / kWaveSize;
  static __device__ __forceinline__ int first_wave(int i) { return i % kPieces * kWavesOfRow; }
  __device__ __forceinline__ void store(const float (&x)[8][8], uint8_t* a, int pitch,
                                        const float* up, uint32_t* lost, const Group& r,
                                        int left) const {
#pragma unroll
    for (int p = 0; p < 8; ++p)
      if (used(p, r, left)) {
        const float f = up[p * kPieces + part];
        half8 h;
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = (_Float16)(x[p][e] * f);
        *reinterpret_cast<half8*>(a + (p * kPieces + part) * pitch + 16 * at) = h;
      }
    float low = 1.0f;
#pragma unroll
    for (int p = 0; p < 8; ++p)
      low = fminf(low, scaled_least(least[p], up[p * kPieces + part]));
    if (low >= kLeast16) return;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      float gone = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) gone += fabsf(lost16(x[p][e] * up[p * kPieces + part]));
      add_lost(&lost[p * kPieces + part], gone);
    }
  }
  __device__ __forceinline__ void store_lost(const float (&x)[8][8], uint8_t* a, int pitch,
                                             const float* up, const Group& r, int left) const {
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      const float f = up[p * kPieces + part];
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = lost_bf16(x[p][2 * i] * f) | lost_bf16(x[p][2 * i + 1] * f) << 16;
      *reinterpret_cast<uint4*>(a + (p * kPieces + part) * pitch + 16 * at) =
          make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
};

template <class Dy, int N, int kWaves>
__global__ __launch_bounds__(kWaves* kWaveSize) void i8_few_gradient_kernel(FewArgs g) {
  constexpr int kThreads = kWaves * kWaveSize;
  constexpr int kDepth = kWaves * kWaveValues / N;  // of A
  constexpr int kPitch = kDepth * 2 + 16;           // bytes of a row of A in LDS
  static_assert(8 * 8 * kThreads == N * kDepth, "every value in one lane");
  __shared__ __attribute__((aligned(16))) uint8_t a[N * kPitch];
  __shared__ uint32_t big[kWaves][N];
  __shared__ float up[N], down[N];
  __shared__ uint32_t lost[N], at_risk[kCols / 16];
  __shared__ uint64_t live[kWaves];  // a bit a column of B that holds more than zeros in a wave's part
  // The steps' stages are apart, so that the compiler can tell a copy into one from a read of
  // another; in each every wave has its own part.
  __shared__ __attribute__((aligned(1024))) uint8_t s0[kWaves * kStepCopy], s1[kWaves * kStepCopy],
      s2[kWaves * kStepCopy], s3[kWaves * kStepCopy], s4[kWaves * kStepCopy];
  uint8_t* const st[NS] = {s0, s1, s2, s3, s4};
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  // neighbours, which share the lines of B, on one XCD
  const int L = xcd_logical_tile(blockIdx.x, gridDim.x);
  const int sg = L / g.tiles, j0 = (L - sg * g.tiles) * kCols;
  const int sp = sg / g.groups, first = (sg - sp * g.groups) * N;
  const Group rows{first, min(N, g.rows - first)};
  const int c0 = sp * g.chunk, left = min(g.depth - c0, g.chunk);  // 1 .. kDepth
  const int nk = (left + kStepRows - 1) / kStepRows, per = (nk + kWaves - 1) / kWaves;
  const int kb = min(nk, wave * per), ke = min(nk, kb + per);

  // Copies: four lanes a row of 64 bytes. Rows past the last are past the end and become
  // zeros, rows of the next split meet zeros of A, columns past the last are not kept; steps
  // past the last copy zeros, without an access of memory, and are not read.
  const __amdgpu_buffer_rsrc_t rb =
      make_rsrc(g.B + j0, (uint32_t)g.depth * (uint32_t)g.cols - (uint32_t)j0);
  const uint32_t at = (uint32_t)(lane >> 2) * (uint32_t)g.cols +
                      16u * (uint32_t)((lane & 3) ^ swz_step(lane >> 2));
  auto issue = [&](uint8_t* stage, int k) __attribute__((always_inline)) {
    uint8_t* mine = stage + wave * kStepCopy;
    const uint32_t so = (uint32_t)(c0 + min(k, nk - 1) * kStepRows) * (uint32_t)g.cols;
    copy16(rb, mine, k < ke ? at : kPastEnd, so);
    copy16(rb, mine + kStepCopy / 2, k < ke ? at + 16u * (uint32_t)g.cols : kPastEnd, so);
  };
  // dY first, all of it at once: loads return in order, and B is much; then the first copies of B,
  // then dY times the scales
  Dy dy;
  auto begin = [&](float (&x)[8][8]) __attribute__((always_inline)) {
    dy.load(g, rows, c0, left);
    asm volatile("" ::: "memory");  // the copies below stay below
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < NS; ++u) issue(st[u], kb + u);
#pragma unroll
    for (int p = 0; p < 8; ++p)
      if (dy.used(p, rows, left)) dy.multiply(x[p], p, left);
  };

  // Lane l takes row l % 16 of A and rows 8 * (l / 16) .. of a step; of eight rows the upper lanes
  // repeat the lower and are not kept.
  const uint8_t* ar = a + (lane & (N - 1)) * kPitch + 16 * (lane >> 4);
  const int kr = 8 * (lane >> 4) + ((lane & 15) >> 1);
  const int bo = wave * kStepCopy + kr * kCols + 8 * (lane & 1), bs = swz_step(kr);
  float4v acc[kCols / 16];
  uint32_t seen[kCols / 16] = {};  // what a column of B holds, one bit over another
  // The wave's part of the contraction, by the left operand, fp16 in LDS, or by what it has lost.
  auto contract = [&](auto second) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < kCols / 16; ++j) acc[j] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
    // tail: -1 where the step issues copies, else how many did not before it
    auto step = [&](uint8_t* stage, int k, auto tail) __attribute__((always_inline)) {
      asm volatile("" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
      // this wave's copies of the step have landed: all but those of the steps behind it
      constexpr int kTail = decltype(tail)::value;
      constexpr int kLeft = 2 * (NS - 1 - (kTail > 0 ? kTail : 0));
      __builtin_amdgcn_s_waitcnt(0x0f70 | (kLeft & 15) | (kLeft >> 4) << 14);
      asm volatile("" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
      const half8 ax = *reinterpret_cast<const half8*>(ar + k * (2 * kStepRows));
      int2v b[kCols / 16];
#pragma unroll
      for (int j = 0; j < kCols / 16; ++j)
        b[j] = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
            (__attribute__((address_space(3))) int2v*)(stage + bo + ((j ^ bs) << 4)));
#pragma unroll
      for (int j = 0; j < kCols / 16; ++j) {
        if constexpr (second) {
          acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              to_bf16s(b[j]), __builtin_bit_cast(bf16x8, ax), acc[j], 0, 0, 0);
        } else {
          seen[j] |= (uint32_t)(b[j][0] | b[j][1]);
          acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(to_halves(b[j]), ax, acc[j], 0, 0, 0);
        }
      }
      if constexpr (kTail >= 0) return;
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
      for (int u = 0; u < NS; ++u) step(st[u], k + u, std::integral_constant<int, -1>{});
    static_assert(NS == 5, "tail");
    if (k < ke) step(s0, k, std::integral_constant<int, 0>{});
    if (k + 1 < ke) step(s1, k + 1, std::integral_constant<int, 1>{});
    if (k + 2 < ke) step(s2, k + 2, std::integral_constant<int, 2>{});
    if (k + 3 < ke) step(s3, k + 3, std::integral_constant<int, 3>{});
    __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0): no copy lands behind this
  };
  // The waves' sums of 16 columns, for one of the first four waves: lane l of a 16 x 16 result holds
  // row l % 16 and four neighbouring columns.
  float4v* sums = reinterpret_cast<float4v*>(a);
  static_assert(kWaves * kCols / 16 * kWaveSize * 16 <= N * kPitch, "sums fit");
  auto exchange = [&]() __attribute__((always_inline)) {
    __syncthreads();  // `a` has been read
#pragma unroll
    for (int j = 0; j < kCols / 16; ++j)
      sums[(wave * (kCols / 16) + j) * kWaveSize + lane] = acc[j];
    __syncthreads();
    const int own = min(wave, kCols / 16 - 1);
    float4v sum = sums[own * kWaveSize + lane];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) sum += sums[(w * (kCols / 16) + own) * kWaveSize + lane];
    return sum;
  };

  // fmaxf passes over NaN: what a row with one is scaled by does not matter.
  {
    float x[8][8];
    begin(x);
    dy.largest(x, rows, left, big[wave]);
    lds_only_barrier();
    if (t < N) {
      uint32_t b = 0;
#pragma unroll
      for (int w = 0; w < Dy::kWavesOfRow; ++w) b = max(b, big[Dy::first_wave(t) + w][t]);
      const PowerOfTwo f = to_fp16_range(b);
      up[t] = f.up;
      down[t] = f.down;
      lost[t] = 0;
    }
    lds_only_barrier();
    dy.store(x, a, kPitch, up, lost, rows, left);
    lds_only_barrier();
  }
  const uint32_t my_lost = lost[lane & (N - 1)];  // row l % N's
  contract(std::false_type{});
  const int n = lane & 15, c = j0 + 16 * wave + 4 * (lane >> 4);
  const bool alive = wave < kCols / 16 && n < rows.count && c < g.cols;
  const bool losing = __any(my_lost != 0);  // the same in all waves
  if (losing) {
    uint64_t columns = 0;
#pragma unroll
    for (int j = 0; j < kCols / 16; ++j) {  // lane l has seen a quarter of column l % 16
      uint64_t m = __ballot(seen[j] != 0);
      m |= m >> 32;
      m |= m >> 16;
      columns |= (m & 0xffffu) << (16 * j);
    }
    if (lane == 0) live[wave] = columns;
  }
  float4v sum = exchange();
  // What the left operand has lost, where a result may rest on it (i8_lost.hpp).
  if (losing) {
    uint64_t columns = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) columns |= live[w];
    const float limit = alive ? lost_limit(my_lost) : 0.0f;
    bool low = false;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      low |= fabsf(sum[e]) < limit && (columns >> ((c - j0 + e) & 63) & 1u);
    const uint64_t mine = __ballot(low);
    if (wave < kCols / 16 && lane == 0) at_risk[wave] = mine != 0;
    lds_only_barrier();
    uint32_t any = 0;
#pragma unroll
    for (int w = 0; w < kCols / 16; ++w) any |= at_risk[w];
    if (__builtin_amdgcn_readfirstlane(any) != 0) {
      {
        float x[8][8];
        begin(x);
        dy.store_lost(x, a, kPitch, up, rows, left);
        lds_only_barrier();
      }
      contract(std::true_type{});
      const float4v more = exchange();
      // of rows at risk in these 16 columns alone, whatever the others hold
      uint64_t row = mine | mine >> 32;
      row |= row >> 16;
      if (row >> n & 1u) sum += more;
    }
  }
  if (!alive) return;
  sum *= down[n];
  if (g.S > 1) {
    *reinterpret_cast<float4v*>(g.part + ((size_t)sp * g.rows + first + n) * g.cols + c) = sum;
    return;
  }
  uint32_t y[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = i8_to_bf16(sum[e]);
  *reinterpret_cast<uint2*>(g.out + (size_t)(first + n) * g.cols + c) =
      make_uint2(y[0] | (y[1] << 16), y[2] | (y[3] << 16));
}

template <template <int, int> class Dy, int N, int WAVES>
void launch(const FewArgs& g, hipStream_t st) {
  hipLaunchKernelGGL((i8_few_gradient_kernel<Dy<N, WAVES * kWaveSize>, N, WAVES>),
                     dim3((unsigned)(g.tiles * g.groups * g.S)), dim3(WAVES * kWaveSize), 0, st, g);
}

}  // namespace

bool plan_i8_few_gradient(I8Plan& p, int rows, int cols, int depth, int splits) {
  const int most = 4 * kWaveValues / (rows <= 8 ? 8 : 16);  // of four waves
  const int S = depth <= 2 * most ? 1 : (depth + most - 1) / most;
  const long long workgroups = (long long)((rows + 15) / 16) * ((cols + kCols - 1) / kCols);
  if (rows > 16 ? S > 1 || workgroups > kGroups : S > splits) return false;
  p.strip = true;
  p.kper = ((depth + S - 1) / S + 63) / 64;  // of 64, at most what a workgroup takes
  p.S = (depth + p.kper * 64 - 1) / (p.kper * 64);
  if (p.S > 1) p.ws_bytes = (size_t)p.S * rows * cols * sizeof(float);
  return true;
}

hipError_t launch_i8_few_gradient(const uint16_t* dY, bool transposed, const float* scale,
                                  const int8_t* B, uint16_t* out, int rows, int cols, int depth,
                                  float* part, const I8Plan& p, hipStream_t st) {
  const FewArgs g{dY,   scale, B,    out, part, rows, depth, cols, (cols + kCols - 1) / kCols,
                  rows <= 8 ? 1 : (rows + 15) / 16, p.S, p.kper * 64};
  if (!transposed)
    rows <= 8 ? launch<Straight, 8, 8>(g, st) : launch<Straight, 16, 8>(g, st);
  else if (rows == 8)
    p.S == 1 ? launch<Transposed, 8, 8>(g, st) : launch<Transposed, 8, 4>(g, st);
  else
    p.S == 1 ? launch<Transposed, 16, 8>(g, st) : launch<Transposed, 16, 4>(g, st);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || p.S == 1) return err;
  return launch_i8_gradient_finish(part, nullptr, out, rows, cols, p.S, st);
}

}  // namespace q4
