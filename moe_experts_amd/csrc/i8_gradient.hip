// Gradients of the 8-bit product:
//   input    dX[m][k] = sum_n (dY[m][n] * sw[n]) * W[n][k]
//   weights  dW[n][k] = sum_m (dY[m][n] * sx[m]) * X[m][k]
// Both are C[i][j] = rs[i] * sum_c A[i][c] * B[c][j] with A fp16 (the bracket, scaled; written
// by a row kernel, for the weights transposed) and B the int8 operand as it stands in memory,
// its rows along the contraction: one kernel on the fp16 matrix cores with fp32 sums. Every
// int8 is an fp16 number, so only A is rounded; what its smallest values lose by it comes back where a
// result may rest on it (i8_lost.hpp).
//
// B's step is copied into LDS as bytes; ds_read_b64_tr_b8 gives a lane eight values of one
// column, that is of the contraction, which become halves in ten instructions: with the
// sign bit turned, a byte behind 0x64 is the half 1024 + 128 + q. Otherwise as the 8-bit
// product's tiles (64 of the contraction a step).
//
// What bounds it: 2048 rows of 4096 x 11008 take 163 to 189 us for the input and 171 to 192 for the
// weights, from GPU to GPU, of which the matrix cores need 75 at the peak clock; the power limit
// holds it at 1.67 to 1.81 and 1.44 to 1.53 GHz call after call. A plain bf16 product of the
// library takes 161 us where these take 163 and 171. The row kernels in front take 22 and 27 us,
// at 4.1 and 5.0 TB/s of what they move.
#include <algorithm>

#include "i8_device.hpp"
#include "i8_internal.hpp"
#include "i8_lost.hpp"
#include "i8_tile.hpp"

namespace q4 {
namespace {

typedef float float16v __attribute__((ext_vector_type(16)));

constexpr int BK = kStepBytes / 2;  // of the contraction in a step

// How a tile goes over the contraction (i8_lost.hpp): by the left operand; the same, looking which
// columns of B hold more than zeros, where a row has lost anything (an instruction for every eight
// values, 1.6 % of a large tile's time); by what the left operand has lost.
enum Pass { kPlain, kLooking, kLost };
template <int P>
using PassTag = std::integral_constant<int, P>;

struct GradArgs {
  const uint16_t* A;  // fp16 [rows][ld]
  const int8_t* B;    // [depth][cols]
  const float* rs;
  const uint16_t* A2;  // bf16 [rows][ld], what A lost, where lost[row] is not 0
  const uint32_t* lost;
  uint16_t* out;      // bf16 [rows][cols]
  int rows, cols, depth, ld;
  int tiles_m, tiles_n, nk, S, kper;
  float* part;
};

// Where 16-byte chunk c of row k stands: eight rows of one chunk, which 16 lanes read at once,
// and their right neighbours, which the next 16 read, meet no bank twice.
template <int BN>
__device__ __forceinline__ int swz_byte(int k) {
  return BN == 256 ? 2 * (k & 7) : 2 * ((k >> 1) & 3);
}

template <int BN, int THREADS>
struct ByteCopy {
  static constexpr int kChunks = BN / 16;
  static constexpr int kInstr = BK * kChunks / THREADS;
  static_assert(THREADS / kChunks % 8 == 0, "one swizzle a lane");
  __amdgpu_buffer_rsrc_t r;
  uint32_t off, pitch;
  __device__ __forceinline__ void init(const GradArgs& g, int j0, int t) {
    pitch = (uint32_t)g.cols;
    // rows past the last are past the end: zeros; columns past the last are not kept
    r = make_rsrc(g.B + j0, (uint32_t)g.depth * pitch - (uint32_t)j0);
    const int k = t / kChunks;
    off = (uint32_t)k * pitch + 16u * (uint32_t)((t % kChunks) ^ swz_byte<BN>(k));
  }
  __device__ __forceinline__ void issue(uint8_t* stage, int ks, bool live, int wave) const {
    const uint32_t so = (uint32_t)ks * BK * pitch;
#pragma unroll
    for (int i = 0; i < kInstr; ++i)
      copy16(r, stage + (i * THREADS + wave * kWaveSize) * 16,
             live ? off + (uint32_t)(i * (THREADS / kChunks)) * pitch : kPastEnd, so);
  }
};

// WAVES a SIMD: what the stages leave room for.
template <int BM, int BN, int WM, int WN, int NS, bool WHOLE, int WAVES>
__global__ __launch_bounds__(WM* WN* kWaveSize, WAVES) void i8_gradient_kernel(GradArgs g) {
  constexpr int kThreads = WM * WN * kWaveSize;
  constexpr int WR = BM / WM, WC = BN / WN;
  constexpr int MI = WR / 32, NJ = WC / 32;
  constexpr int kA = BM * kStepBytes, kB = BK * BN, kStage = kA + kB;
  constexpr int kPitch = WC * 2 + 16;
  // The steps' stages are apart, so that the compiler can tell a copy into one from a read of
  // another.
  __shared__ __attribute__((aligned(1024))) uint8_t s0[kStage], s1[kStage];
  __shared__ __attribute__((aligned(1024))) uint8_t s2[NS > 2 ? kStage : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t s3[NS > 3 ? kStage : 16];
  uint8_t* const st[4] = {s0, s1, s2, s3};
  const int L = xcd_logical_tile(blockIdx.x, gridDim.x);
  const int tiles = g.tiles_m * g.tiles_n;
  const int sp = L / tiles;
  int tm, tn;
  tile_of(L - sp * tiles, g.tiles_m, g.tiles_n, tm, tn);
  const int i0 = tm * BM, j0 = tn * BN;
  const int rows = min(BM, g.rows - i0);
  const int kb = sp * g.kper, ke = min(g.nk, kb + g.kper);
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = wave % WM, wn = wave / WM;

  RowCopy<BM, kThreads> ca;
  ByteCopy<BN, kThreads> cb;
  ca.init(g.A + (size_t)i0 * g.ld, rows, (uint32_t)g.ld * 2u, t);
  cb.init(g, j0, t);
  constexpr int kCopies = ca.kInstr + cb.kInstr;  // of a wave in a step

  float16v acc[MI][NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
  struct Operands {
    half8 a[MI];  // or the bits of bf16 numbers
    int2v b[NJ];
  };
  const int ra = wm * WR + (lane & 31);
  const int ao = ra * kStepBytes + (((lane >> 5) ^ swz_row(ra)) << 4);
  // The 16 lanes of a group read eight rows of 16 columns; lane l gets column l % 32 of the
  // wave's 32, rows 8 * (l / 32) .. of the quarter's 16.
  const int kr = 8 * (lane >> 5) + ((lane & 15) >> 1);
  const int bo = kA + kr * BN + 8 * (lane & 1);
  const int bc = wn * (WC / 16) + ((lane >> 4) & 1);
  const int bs = swz_byte<BN>(kr);
  auto read = [&](Operands& o, const uint8_t* stage, int q) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
      o.a[i] = *reinterpret_cast<const half8*>(stage + (ao ^ (q << 5)) + 32 * i * kStepBytes);
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      o.b[j] = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
          (__attribute__((address_space(3))) int2v*)(stage + bo + q * 16 * BN +
                                                     (((bc + 2 * j) ^ bs) << 4)));
  };
  uint32_t live[NJ] = {};  // what a column of B holds, one bit over another
  auto multiply = [&](const Operands& o, auto pass) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      if constexpr (pass == kLooking) live[j] |= (uint32_t)(o.b[j][0] | o.b[j][1]);
      if constexpr (pass == kLost) {
        const bf16x8 b = to_bf16s(o.b[j]);
#pragma unroll
        for (int i = 0; i < MI; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
              b, __builtin_bit_cast(bf16x8, o.a[i]), acc[i][j], 0, 0, 0);
      } else {
        const half8 b = to_halves(o.b[j]);
#pragma unroll
        for (int i = 0; i < MI; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(b, o.a[i], acc[i][j], 0, 0, 0);
      }
    }
  };
  // whether a row of the tile has lost anything; loads return in order, so that nothing is waited
  // for that the first products do not need
  uint32_t lost = 0;
#pragma unroll
  for (int i = 0; i < BM; i += kWaveSize) lost |= g.lost[min(i0 + i + lane, g.rows - 1)];
  asm volatile("" ::: "memory");  // the copies below stay below
  __builtin_amdgcn_sched_barrier(0);
  // steps past the last copy zeros, without an access of memory, and are not read
  auto issue = [&](const RowCopy<BM, kThreads>& left, uint8_t* stage, int ks)
                   __attribute__((always_inline)) {
    const int k = min(ks, ke - 1);
    left.issue(stage, k, ks < ke ? kStepBytes : 0, wave);  // ld is whole steps
    cb.issue(stage + kA, k, ks < ke, wave);
  };
  auto begin = [&](const RowCopy<BM, kThreads>& left) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < NS; ++u) issue(left, st[u], kb + u);
  };
  // the contraction from kb to ke, behind begin()
  constexpr int Q = BK / 16;
  auto contract = [&](const RowCopy<BM, kThreads>& left, auto pass)
                      __attribute__((always_inline)) {
    Operands o[WHOLE ? 2 * Q : 2];
    auto step = [&](uint8_t* cur, uint8_t* next, int ks, int half) __attribute__((always_inline)) {
      if constexpr (WHOLE) {
        tile_hand_over<kCopies*(NS - 2)>();
#pragma unroll
        for (int q = 0; q < Q; ++q) read(o[Q * (1 - half) + q], next, q);
        issue(left, cur, ks + NS);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int q = 0; q < Q; ++q) multiply(o[Q * half + q], pass);
        __builtin_amdgcn_sched_barrier(0);
      } else {
#pragma unroll
        for (int q = 0; q < Q - 1; ++q) {
          read(o[(q + 1) & 1], cur, q + 1);
          __builtin_amdgcn_sched_barrier(0);
          multiply(o[q & 1], pass);
          __builtin_amdgcn_sched_barrier(0);
        }
        tile_hand_over<kCopies*(NS - 2)>();
        read(o[0], next, 0);
        issue(left, cur, ks + NS);
        __builtin_amdgcn_sched_barrier(0);
        multiply(o[1], pass);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    tile_hand_over<kCopies*(NS - 1)>();
#pragma unroll
    for (int q = 0; q < (WHOLE ? Q : 1); ++q) read(o[q], s0, q);
    // stages and operand sets alternate at compile time
    constexpr int U = WHOLE && NS % 2 ? 2 * NS : NS;
    int ks = kb;
    for (; ks + U <= ke; ks += U)
#pragma unroll
      for (int u = 0; u < U; ++u) step(st[u % NS], st[(u + 1) % NS], ks + u, u & 1);
#pragma unroll
    for (int u = 0; u < U - 1; ++u)
      if (ks + u < ke) step(st[u % NS], st[(u + 1) % NS], ks + u, u & 1);
    tile_hand_over<0>();  // the last copies have landed before their places are used again
  };
  begin(ca);
  const bool losing = __any(lost != 0);  // the same in all waves
  if (losing)
    contract(ca, PassTag<kLooking>{});
  else
    contract(ca, PassTag<kPlain>{});

  // Lane l holds row l % 32 of A, register r column 8 * (r / 4) + 4 * (l / 32) + r % 4.
  const int iw = i0 + wm * WR, rlive = rows - wm * WR;
  const int jw = j0 + wn * WC;
  const int lr = lane & 31, l4 = 4 * (lane >> 5);
  // What the left operand has lost, where a result may rest on it (i8_lost.hpp): all waves of the
  // workgroup agree on the rows, a bit each.
  if (losing) {
    __shared__ uint32_t at_risk[WN][BM / 32];
    uint32_t low[MI][NJ];  // a bit a result
    uint32_t any_low = 0;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const float limit =
          32 * i + lr < rlive ? lost_limit(g.lost[min(iw + 32 * i + lr, g.rows - 1)]) : 0.0f;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        low[i][j] = 0;
#pragma unroll
        for (int r = 0; r < 16; ++r)
          low[i][j] |= fabsf(acc[i][j][r]) < limit ? 1u << r : 0u;
        // held as bits, not as a mask of lanes for every result
        asm volatile("" : "+v"(low[i][j]));
        any_low |= low[i][j];
      }
    }
    uint32_t rows_low[MI] = {};
    if (__any(any_low != 0)) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        // unless their columns are zeros, or none of the result's: lane l has seen half of
        // column l % 32
        const uint64_t seen = __ballot(live[j] != 0);
        const int left = g.cols - (jw + 32 * j);
        const uint32_t in = left <= 0 ? 0u : left < 32 ? (1u << left) - 1u : ~0u;
        const uint32_t columns = (((uint32_t)seen | (uint32_t)(seen >> 32)) & in) >> l4;
        // the columns of a lane's results, in the order of its registers
        const uint32_t own = (columns & 15u) | (columns >> 4 & 0xf0u) | (columns >> 8 & 0xf00u) |
                             (columns >> 12 & 0xf000u);
#pragma unroll
        for (int i = 0; i < MI; ++i) {
          const uint64_t lanes = __ballot((low[i][j] & own) != 0);
          rows_low[i] |= (uint32_t)lanes | (uint32_t)(lanes >> 32);
        }
      }
    }
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < MI; ++i) at_risk[wn][wm * MI + i] = rows_low[i];
    lds_only_barrier();
    uint32_t any = 0;
#pragma unroll
    for (int w = 0; w < WN; ++w)
#pragma unroll
      for (int i = 0; i < BM / 32; ++i) any |= at_risk[w][i];
    if (__builtin_amdgcn_readfirstlane(any) != 0) {
      RowCopy<BM, kThreads> c2;
      c2.init(g.A2 + (size_t)i0 * g.ld, rows, (uint32_t)g.ld * 2u, t);
#pragma unroll
      for (int i = 0; i < c2.kInstr; ++i) {
        const int row = (i * kThreads + t) / c2.kChunks;
        uint32_t bits = 0;
#pragma unroll
        for (int w = 0; w < WN; ++w) bits |= at_risk[w][row >> 5];
        if (!(bits >> (row & 31) & 1u)) c2.off[i] = kPastEnd;
      }
      begin(c2);
      contract(c2, PassTag<kLost>{});
    }
  }
  if (g.S > 1) {
    float* dst = g.part + (size_t)sp * g.rows * g.cols;
#pragma unroll
    for (int i = 0; i < MI; ++i)
      if (32 * i + lr < rlive)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int n = jw + 32 * j + 8 * q + l4;
            if (n < g.cols)
              *reinterpret_cast<float4*>(dst + (size_t)(iw + 32 * i + lr) * g.cols + n) =
                  make_float4(acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                              acc[i][j][4 * q + 3]);
          }
    return;
  }
  constexpr int kFit = kStage / (32 * kPitch);  // waves whose results fit a stage
  static_assert(kFit * NS >= WM * WN, "results fit the stages");
  uint8_t* res = s0;
#pragma unroll
  for (int u = 1; u < NS; ++u)
    if (wave / kFit == u) res = st[u];
  res += wave % kFit * (32 * kPitch);
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const float s = g.rs[min(iw + 32 * i + lr, g.rows - 1)];
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t e[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) e[u] = i8_to_bf16(acc[i][j][4 * q + u] * s);
        *reinterpret_cast<uint2*>(res + lr * kPitch + (32 * j + 8 * q + l4) * 2) =
            make_uint2(e[0] | (e[1] << 16), e[2] | (e[3] << 16));
      }
    constexpr int kPieces = WC / 8;
#pragma unroll
    for (int p0 = 0; p0 < 32 * kPieces; p0 += kWaveSize) {
      const int r = (p0 + lane) / kPieces, pc = (p0 + lane) % kPieces;
      const int n = jw + 8 * pc;
      if (32 * i + r < rlive && n < g.cols)
        *reinterpret_cast<uint4*>(g.out + (size_t)(iw + 32 * i + r) * g.cols + n) =
            *reinterpret_cast<const uint4*>(res + r * kPitch + 16 * pc);
    }
  }
}

template <int BM, int BN, int WM, int WN, int NS, bool WHOLE, int WAVES>
void launch_tile(const GradArgs& g, hipStream_t st) {
  hipLaunchKernelGGL((i8_gradient_kernel<BM, BN, WM, WN, NS, WHOLE, WAVES>),
                     dim3((unsigned)(g.tiles_m * g.tiles_n * g.S)), dim3(WM * WN * kWaveSize), 0,
                     st, g);
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

// Tiles, measured (us a call on the GPU, with the row kernel): 11008 x 4096 results over 2048:
// 128 x 256 211, 128 x 128 214; 2048 x 4096 over 11008: 195, 203; 1536 x 5120 over 777: 27.2, 27.6,
// and 64 x 128 31.3; 150 x 11008 over 4096: 128 x 128 39.8, 64 x 128 39.9, 32 x 128 30.8; 130 x 4096
// over 4096: 128 x 128 in 4 splits 24.8, 64 x 128 in 2 23.4, 32 x 128 22.2. Two stages do better
// than more where two workgroups fit a CU by that: 128 x 256 in 3 stages 219 instead of 190, the
// product alone.
constexpr I8Tile kTiles[] = {{128, 256, 0.80, 0.72, 0.25},
                             {128, 128, 0.30, 0.28, 0.27},
                             {64, 128, 0.26, 0.20, 0.12},
                             {32, 128, 0.18, 0.10, 0.09}};

// rows x cols results over a contraction of `depth`; chunks of `big` for the transposition
I8Plan plan_gradient(int rows, int cols, int depth, int chunks) {
  I8Plan p{};
  p.ld = (depth + BK - 1) / BK * BK;
  plan_i8_tiles(p, kTiles, rows, cols, p.ld / BK);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at = align256(at + bytes);
    return o;
  };
  p.off_a = take((size_t)rows * p.ld * 2);
  p.off_a2 = take((size_t)rows * p.ld * 2);
  p.off_rs = take((size_t)rows * sizeof(float));
  p.off_lost = take((size_t)rows * sizeof(uint32_t));
  p.off_max = take((size_t)2 * chunks * rows * sizeof(uint32_t));
  p.off_part = take(p.S > 1 ? (size_t)p.S * rows * cols * sizeof(float) : 0);
  p.ws_bytes = at;
  return p;
}

LeftOperand left_operand(uint8_t* w, const I8Plan& p) {
  return {reinterpret_cast<uint16_t*>(w + p.off_a), reinterpret_cast<uint16_t*>(w + p.off_a2),
          reinterpret_cast<float*>(w + p.off_rs), reinterpret_cast<uint32_t*>(w + p.off_lost), p.ld};
}

hipError_t launch_tiles(const int8_t* B, uint16_t* out, int rows, int cols, int depth, uint8_t* w,
                        const I8Plan& p, hipStream_t st) {
  if ((long long)p.tiles_m * p.tiles_n * p.S > 0x3fffffLL) return hipErrorInvalidValue;
  const LeftOperand l = left_operand(w, p);
  GradArgs g{l.a,
             B,
             l.rs,
             l.a2,
             l.lost,
             out,
             rows,
             cols,
             depth,
             p.ld,
             p.tiles_m,
             p.tiles_n,
             p.nk,
             p.S,
             p.kper,
             reinterpret_cast<float*>(w + p.off_part)};
  switch (p.tile) {
    case 0: launch_tile<128, 256, 2, 4, 2, false, 4>(g, st); break;
    case 1: launch_tile<128, 128, 2, 4, 2, false, 6>(g, st); break;
    case 2: launch_tile<64, 128, 2, 4, 4, true, 4>(g, st); break;
    default: launch_tile<32, 128, 1, 4, 4, true, 3>(g, st);
  }
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || p.S == 1) return err;
  return launch_i8_gradient_finish(g.part, g.rs, out, rows, cols, p.S, st);
}

}  // namespace

I8Plan plan_i8_backward(int M, int N, int K) {
  I8Plan p{};
  if (plan_i8_few_gradient(p, M, K, N, 1)) return p;
  return plan_gradient(M, K, N, 0);
}

I8RowsPlan plan_i8_backward_rows(int M, int N, int K) {
  const I8Plan p = plan_i8_backward(M, N, K);
  return p.strip ? I8RowsPlan{} : plan_i8_gradient_rows(p.ld);
}

hipError_t launch_i8_backward(const uint16_t* dY, const int8_t* W, const float* sw, uint16_t* dX,
                              int M, int N, int K, void* ws, const I8Plan& p, hipStream_t st) {
  if (p.strip) return launch_i8_few_gradient(dY, false, sw, W, dX, M, K, N, nullptr, p, st);
  uint8_t* w = static_cast<uint8_t*>(ws);
  const hipError_t err = launch_i8_gradient_rows(dY, sw, left_operand(w, p), M, N, st);
  if (err != hipSuccess) return err;
  return launch_tiles(W, dX, M, K, N, w, p, st);
}

I8Plan plan_i8_backward_weight(int M, int N, int K) {
  I8Plan p{};
  if (plan_i8_few_gradient(p, N, K, M, kFewSplits)) return p;
  return plan_gradient(N, K, M, i8_max_chunks(M, N));
}

I8RowsPlan plan_i8_backward_weight_rows(int M, int N, int K) {
  const I8Plan p = plan_i8_backward_weight(M, N, K);
  return p.strip ? I8RowsPlan{} : plan_i8_gradient_columns(M, N, p.ld);
}

hipError_t launch_i8_backward_weight(const uint16_t* dY, const int8_t* X, const float* sx,
                                     uint16_t* dW, int M, int N, int K, void* ws, const I8Plan& p,
                                     hipStream_t st) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  if (p.strip)
    return launch_i8_few_gradient(dY, true, sx, X, dW, N, K, M, reinterpret_cast<float*>(w), p, st);
  const hipError_t err = launch_i8_gradient_columns(
      dY, sx, left_operand(w, p), reinterpret_cast<uint32_t*>(w + p.off_max), M, N, st);
  if (err != hipSuccess) return err;
  return launch_tiles(X, dW, N, K, M, w, p, st);
}

}  // namespace q4
