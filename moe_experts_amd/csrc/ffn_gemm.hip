// Prompt and gradient GEMMs of the dense feed-forward operators over Q4_0
// weights, on the fp16 matrix cores with fp32 sums:
//   dual      H = act(X . deq(Wg)) * (X . deq(Wu))            X fp16 [M][K]
//   adapters  Y = X . deq(B) + t . B_id^T                     X fp16 [M][K]
//   gradient  dX = dG . deq(Wg)^T + dU . deq(Wu)^T            one or two matrices
//
// Tile BM x 128, K steps of 64, 512 lanes: 4 consumer waves issue only matrix
// instructions, 4 producer waves fetch the weights, dequantize them into an
// fp16 LDS tile [column][k] and issue the copies of the left operand, so the
// VALU work of one role runs beside the matrix work of the other.
//
//   * Left operand: 16-byte LDS-DMA copies, three steps deep, issued two steps
//     ahead, XOR-swizzled on the source side.
//   * Weights: a producer lane loads its own share of a step straight into
//     registers, two steps ahead, and writes the dequantized values into the
//     double-buffered LDS tile one step ahead. The raw bytes never pass
//     through LDS.
//   * dual: the 128 columns of a tile are 64 columns of the gate and the same
//     64 of the up matrix, in blocks gate, up, gate, up, so that the wave that
//     holds a column's gate holds its up value in the same lane and register,
//     and the product costs no exchange.
//   * gradient: column c of the result is row c of the weights, whose blocks
//     run along the contraction. A dword of nibbles is then eight values of k
//     of one column, and masking it with 0x000f000f at shifts 0, 4, 8, 12
//     gives the pairs (0,4) (1,5) (2,6) (3,7): the left operand is stored in
//     that order, so nothing is moved. Both matrices form one contraction of
//     2N: steps past the first matrix read the second.
//   * few rows: the contraction is split over workgroups (fp32 partial sums,
//     added in split order by a second kernel), so that the grid fills the GPU.
//
// Each dequantized weight (q - 8) * d is rounded to fp16 before its product,
// as in q4_0_gemm; the sums are fp32.
#include <type_traits>

#include "ffn_device.hpp"
#include "ffn_internal.hpp"
#include "q4_device.hpp"

namespace q4 {
namespace {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef float float16v __attribute__((ext_vector_type(16)));

constexpr int BN = 128, BK = 64;
constexpr int kRole = 256;                 // lanes of one role
constexpr int kXStages = 3;
constexpr int kColBytes = BK * 2;          // one column or row of a step in LDS
constexpr int kBBytes = BN * kColBytes;    // 16 KiB
constexpr uint32_t kOut = 0x80000000u;

enum Side { kAdapters, kDual, kGradient };

struct TileArgs {
  const uint16_t* X;      // left operand [M][lda]
  const uint8_t* W0;
  const uint8_t* W1;      // up matrix, or the second matrix of a gradient
  int M, ncols, lda;      // ncols: columns of one result
  int NB, wrows;          // blocks of a weight row, weight rows
  int tiles_n, S, kper, nk;
  int nk_mat;             // gradient: steps of one matrix
  float* part;            // S > 1: [mats][S][M][ncols]
  // results when S == 1
  _Float16 *H, *G, *U;    // dual: h and, unless null, g and u; adapters: H is Y
  int act;
  const _Float16* t16;    // adapters
  const float* ts;
  Adapters ad;
  uint16_t* dX;           // gradient
  const float* rs;
};

__device__ __forceinline__ int swz_x(int r) { return (r >> 1) & 7; }
__device__ __forceinline__ int swz_b(int n) { return ((n >> 1) ^ (n >> 5)) & 7; }

__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Constants of the dequantization. The mask is kept in a vector register, so
// that masking and setting the exponent is one instruction (which takes at
// most one constant from elsewhere).
struct Dequant {
  uint32_t mask = 0x000f000fu;
  __device__ __forceinline__ Dequant() { asm volatile("" : "+v"(mask)); }
  __device__ __forceinline__ half2v pair(uint32_t nibbles, half2v d) const {
    // binary16 0x6400 | v is 1024 + v exactly; (q - 8) is exact, the product is rounded once
    const half2v off = {(_Float16)1032.0f, (_Float16)1032.0f};
    return (__builtin_bit_cast(half2v, (nibbles & mask) | 0x64006400u) - off) * d;
  }
};

// An 8-byte LDS store that the compiler does not order after the LDS copies in
// flight (written as an assignment it waited for all of them, though they go to
// another array). The barrier after it waits for it (lgkmcnt).
__device__ __forceinline__ void lds_store8(uint8_t* p, uint2 v) {
  const uint32_t at =
      (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)p;
  asm volatile("ds_write_b64 %0, %1" ::"v"(at), "v"(__builtin_bit_cast(uint64_t, v)) : "memory");
}

// ---------------------------------------------------------------- weights
// Forward: the step's 64 weight rows x 128 columns are 256 units of 4 rows x 8
// columns, one a producer lane. Lane l of producer wave w: dword c = l % 8 of
// the column half w / 2 (block c / 4, dword c % 4), rows 4 * rg .. + 3 with
// rg = l / 8 + 8 * (w % 2). dual: half 0 is the gate, half 1 the up matrix.
template <bool DUAL>
struct ForwardWeights {
  static constexpr int kLoads = 8;
  __amdgpu_buffer_rsrc_t r;
  Dequant dq;
  uint32_t vq, vd, pitch;
  uint32_t st;  // LDS byte offset of column 0 of the unit, before the swizzle
  int n0, chunk, half;
  struct Raw {
    uint32_t q[4], d[4];
  };
  __device__ __forceinline__ void init(const TileArgs& g, int tn, int t) {
    const int w = __builtin_amdgcn_readfirstlane(t >> 6);
    const int l = t & 63;
    const int hw = w >> 1;
    const int c = l & 7, rg = (l >> 3) + 8 * (w & 1);
    const int blk = c >> 2, quarter = c & 3;
    pitch = (uint32_t)g.NB * kBlockBytes;
    const uint8_t* base = (DUAL && hw) ? g.W1 : g.W0;
    r = make_rsrc(base, (uint32_t)g.wrows * pitch);
    const int col = DUAL ? 2 * tn + blk : 4 * tn + 2 * hw + blk;  // block column
    // a block column past the matrix reads zeros
    const uint32_t o = (uint32_t)(4 * rg) * pitch + (uint32_t)col * kBlockBytes;
    vd = col < g.NB ? o : kOut;
    vq = col < g.NB ? o + 2 + 4 * quarter : kOut;
    n0 = (DUAL ? 2 * blk + hw : 2 * hw + blk) * 32 + quarter * 8;
    chunk = rg >> 1;
    half = rg & 1;
  }
  __device__ __forceinline__ void load(Raw& raw, int ks) const {
    const uint32_t so = (uint32_t)ks * (BK * pitch);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      raw.q[i] = __builtin_amdgcn_raw_buffer_load_b32(r, vq, so + i * pitch, 0);
      raw.d[i] = __builtin_amdgcn_raw_buffer_load_b16(r, vd, so + i * pitch, 0);
    }
  }
  __device__ __forceinline__ void store(const Raw& raw, uint8_t* __restrict__ bs) const {
    const half2v d01 = __builtin_bit_cast(half2v, (raw.d[0] & 0xffffu) | (raw.d[1] << 16));
    const half2v d23 = __builtin_bit_cast(half2v, (raw.d[2] & 0xffffu) | (raw.d[3] << 16));
    // columns 0..3 sit in the low halves of the rows' dwords, 4..7 in the high ones
    const uint32_t p01[2] = {__builtin_amdgcn_perm(raw.q[1], raw.q[0], 0x05040100u),
                             __builtin_amdgcn_perm(raw.q[1], raw.q[0], 0x07060302u)};
    const uint32_t p23[2] = {__builtin_amdgcn_perm(raw.q[3], raw.q[2], 0x05040100u),
                             __builtin_amdgcn_perm(raw.q[3], raw.q[2], 0x07060302u)};
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const int sh = 4 * (c & 3);
      uint2 v;
      v.x = __builtin_bit_cast(uint32_t, dq.pair(p01[c >> 2] >> sh, d01));
      v.y = __builtin_bit_cast(uint32_t, dq.pair(p23[c >> 2] >> sh, d23));
      const int n = n0 + c;
      lds_store8(bs + n * kColBytes + ((chunk ^ swz_b(n)) << 4) + half * 8, v);
    }
  }
};

// Gradient: the step's tile is 128 weight rows x 2 blocks, one block a
// producer lane (row t / 2, block t % 2).
struct GradientWeights {
  static constexpr int kLoads = 2;
  __amdgpu_buffer_rsrc_t r0, r1;
  Dequant dq;
  uint32_t vq, vd;
  int nk_mat, n, b;
  struct Raw {
    uint32_t q[4], d;
  };
  __device__ __forceinline__ void init(const TileArgs& g, int tn, int t) {
    n = t >> 1;
    b = t & 1;
    const uint32_t pitch = (uint32_t)g.NB * kBlockBytes;
    const int c0 = tn * BN;
    // rows past the matrix read zeros
    const uint32_t bytes = (uint32_t)min(BN, g.wrows - c0) * pitch;
    r0 = make_rsrc(g.W0 + (size_t)c0 * pitch, bytes);
    r1 = make_rsrc((g.W1 ? g.W1 : g.W0) + (size_t)c0 * pitch, bytes);
    vd = (uint32_t)n * pitch + (uint32_t)b * kBlockBytes;
    vq = vd + 2;
    nk_mat = g.nk_mat;
  }
  __device__ __forceinline__ void load(Raw& raw, int ks) const {
    const bool second = ks >= nk_mat;
    const uint32_t so = (uint32_t)(second ? ks - nk_mat : ks) * (2 * kBlockBytes);
    const __amdgpu_buffer_rsrc_t r = second ? r1 : r0;
    const auto v = __builtin_amdgcn_raw_buffer_load_b128(r, vq, so, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) raw.q[i] = v[i];
    raw.d = __builtin_amdgcn_raw_buffer_load_b16(r, vd, so, 0);
  }
  __device__ __forceinline__ void store(const Raw& raw, uint8_t* __restrict__ bs) const {
    const half2v d = __builtin_bit_cast(half2v, (raw.d & 0xffffu) | (raw.d << 16));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint4 v;
      v.x = __builtin_bit_cast(uint32_t, dq.pair(raw.q[i], d));
      v.y = __builtin_bit_cast(uint32_t, dq.pair(raw.q[i] >> 4, d));
      v.z = __builtin_bit_cast(uint32_t, dq.pair(raw.q[i] >> 8, d));
      v.w = __builtin_bit_cast(uint32_t, dq.pair(raw.q[i] >> 12, d));
      *reinterpret_cast<uint4*>(bs + n * kColBytes + (((4 * b + i) ^ swz_b(n)) << 4)) = v;
    }
  }
};

// ---------------------------------------------------------------- left operand
template <int BM>
struct LeftCopies {
  static constexpr int kInstr = BM * kColBytes / 16 / kRole;
  __amdgpu_buffer_rsrc_t r;
  uint32_t off[kInstr], wslot;
  __device__ __forceinline__ void init(const TileArgs& g, int m0, int rows, int t) {
    r = make_rsrc(g.X + (size_t)m0 * g.lda, (uint32_t)rows * (uint32_t)g.lda * 2u);
    wslot = (uint32_t)__builtin_amdgcn_readfirstlane(t >> 6) * (kWaveSize * 16);
#pragma unroll
    for (int i = 0; i < kInstr; ++i) {
      const int slot = i * kRole + t;
      const int row = slot >> 3;
      const int c = (slot & 7) ^ swz_x(row);
      off[i] = row < rows ? ((uint32_t)row * (uint32_t)g.lda + 8u * c) * 2u : kOut;
    }
  }
  __device__ __forceinline__ void issue(uint8_t* __restrict__ stage, int ks) const {
#pragma unroll
    for (int i = 0; i < kInstr; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_t*)(stage + wslot + i * kRole * 16),
                                               16, off[i], (uint32_t)ks * kColBytes, 0, 0);
  }
};

// What the producers do while step ks is multiplied: issue the copies of ks + 2,
// dequantize ks + 1 from its registers into its LDS tile, load ks + 3 into them.
template <int BM, class W>
__device__ __forceinline__ void produce_step(const W& wt, const LeftCopies<BM>& left,
                                             typename W::Raw& raw, uint8_t* __restrict__ xs,
                                             uint8_t* __restrict__ b, int& xst, int ks, int ke) {
  left.issue(xs + xst * (BM * kColBytes), min(ks + 2, ke - 1));
  xst = xst == kXStages - 1 ? 0 : xst + 1;
  __builtin_amdgcn_sched_barrier(0);
  wt.store(raw, b);
  __builtin_amdgcn_sched_barrier(0);
  wt.load(raw, min(ks + 3, ke - 1));
  __builtin_amdgcn_sched_barrier(0);
  // the left operand of ks + 1 landed; what was issued after it may be in flight
  constexpr int kAfter = 2 * W::kLoads + LeftCopies<BM>::kInstr;
  static_assert(kAfter < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt(vmcnt_imm(kAfter) & ~0x0f00);
  lds_barrier();
}

// The producer waves (lane t of them) over the K steps [kb, ke). Steps past the
// last repeat it: they land in a stage that is not read.
template <int BM, Side SIDE>
__device__ __forceinline__ void produce(const TileArgs& g, uint8_t* __restrict__ xs,
                                        uint8_t* __restrict__ bs, int m0, int rows, int tn, int kb, int ke, int t) {
  using W = typename std::conditional<SIDE == kGradient, GradientWeights,
                                      ForwardWeights<SIDE == kDual>>::type;
  constexpr int kXBytes = BM * kColBytes;
  W wt;
  wt.init(g, tn, t);
  LeftCopies<BM> left;
  left.init(g, m0, rows, t);
  typename W::Raw raw[2];
  wt.load(raw[0], kb);
  __builtin_amdgcn_sched_barrier(0);
  left.issue(xs, kb);
  __builtin_amdgcn_sched_barrier(0);
  wt.load(raw[1], min(kb + 1, ke - 1));
  __builtin_amdgcn_sched_barrier(0);
  left.issue(xs + kXBytes, min(kb + 1, ke - 1));
  __builtin_amdgcn_sched_barrier(0);
  wt.store(raw[0], bs);
  __builtin_amdgcn_sched_barrier(0);
  wt.load(raw[0], min(kb + 2, ke - 1));
  __builtin_amdgcn_sched_barrier(0);
  // left operand of step kb landed; everything issued after it may be in flight
  constexpr int kAfter = 2 * W::kLoads + LeftCopies<BM>::kInstr;
  __builtin_amdgcn_s_waitcnt(vmcnt_imm(kAfter) & ~0x0f00);
  lds_barrier();
  int xst = 2;  // stage of the copies two steps ahead
  int ks = kb;
  for (; ks + 2 <= ke; ks += 2) {
    produce_step<BM>(wt, left, raw[1], xs, bs + kBBytes, xst, ks, ke);
    produce_step<BM>(wt, left, raw[0], xs, bs, xst, ks + 1, ke);
  }
  if (ks < ke) produce_step<BM>(wt, left, raw[1], xs, bs + kBBytes, xst, ks, ke);
  __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));  // no copy lands after the workgroup ends
}

template <int BM, Side SIDE>
__global__ __launch_bounds__(2 * kRole, BM == 64 ? 4 : 2) void ffn_gemm_kernel(TileArgs g) {
  constexpr int kXBytes = BM * kColBytes;
  __shared__ __attribute__((aligned(1024))) uint8_t xs[kXStages * kXBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t bs[2 * kBBytes];
  const int L = xcd_logical_tile(blockIdx.x, gridDim.x);
  const int tn = L % g.tiles_n;
  const int rest = L / g.tiles_n;
  const int sp = rest % g.S;
  const int tm = rest / g.S;
  const int m0 = tm * BM;
  const int rows = min(BM, g.M - m0);
  const int kb = sp * g.kper;
  const int ke = min(g.nk, kb + g.kper);  // kb < ke: the plan leaves no split empty
  const int wave = threadIdx.x >> 6;

  if (wave >= 4) {
    produce<BM, SIDE>(g, xs, bs, m0, rows, tn, kb, ke, (int)threadIdx.x - kRole);
    return;
  }

  // -------------------------------------------------------------- consumer
  const int lane = threadIdx.x & 63;
  constexpr int WGR = BM == 256 ? 4 : 2;  // waves along the rows
  constexpr int WR = BM / WGR;            // rows of a wave: 64 or 32
  constexpr int WC = BN / (4 / WGR);      // columns of a wave: 128 or 64
  constexpr int MI = WR / 32, NJ = WC / 32;
  const int wm = wave % WGR;
  const int wn = wave / WGR;
  float16v acc[MI][NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
  lds_barrier();
  int xst = 0;
  for (int ks = kb; ks < ke; ++ks) {
    const uint8_t* x = xs + xst * kXBytes;
    xst = xst == kXStages - 1 ? 0 : xst + 1;
    const uint8_t* b = bs + ((ks - kb) & 1) * kBBytes;
#pragma unroll
    for (int kk = 0; kk < BK / 16; ++kk) {
      const int kc = 2 * kk + (lane >> 5);
      half8 af[MI], bf[NJ];
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const int r = wm * WR + i * 32 + (lane & 31);
        af[i] = *reinterpret_cast<const half8*>(x + r * kColBytes + ((kc ^ swz_x(r)) << 4));
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int n = wn * WC + j * 32 + (lane & 31);
        bf[j] = *reinterpret_cast<const half8*>(b + n * kColBytes + ((kc ^ swz_b(n)) << 4));
      }
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(af[i], bf[j], acc[i][j], 0, 0, 0);
    }
    __builtin_amdgcn_s_waitcnt(0xc07f);  // this wave's reads done before the stages are reused
    lds_barrier();
  }

  // A 32 x 32 fp32 result: lane l holds column l % 32; register r holds row
  // 8 * (r / 4) + 4 * (l / 32) + r % 4.
  const int mw = m0 + wm * WR;     // first row of the wave
  const int rw = rows - wm * WR;   // its live rows
  auto row_of = [&](int i, int r) { return i * 32 + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3); };

  if (g.S > 1) {
    const size_t slab = (size_t)g.M * g.ncols;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int v = wn * WC + j * 32;  // column of the tile
      const int mat = SIDE == kDual ? (v >> 5) & 1 : 0;
      const int col = (SIDE == kDual ? tn * 64 + (v >> 6) * 32 : tn * BN + v) + (lane & 31);
      if (col >= g.ncols) continue;
      float* dst = g.part + ((size_t)mat * g.S + sp) * slab + col;
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (row_of(i, r) < rw) dst[(size_t)(mw + row_of(i, r)) * g.ncols] = acc[i][j][r];
    }
    return;
  }

  if constexpr (SIDE == kDual) {
#pragma unroll
    for (int j = 0; j < NJ; j += 2) {
      const int col = tn * 64 + (wn * WC / 64 + j / 2) * 32 + (lane & 31);
      if (col >= g.ncols) continue;
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          if (row_of(i, r) >= rw) continue;
          const size_t o = (size_t)(mw + row_of(i, r)) * g.ncols + col;
          const float gt = acc[i][j][r], up = acc[i][j + 1][r];
          g.H[o] = (_Float16)(act_value(gt, g.act) * up);
          if (g.G) {
            g.G[o] = (_Float16)gt;
            g.U[o] = (_Float16)up;
          }
        }
    }
  } else if constexpr (SIDE == kAdapters) {
    // Wide half of the adapters: for every adapter that occurs in the wave's
    // rows, t16 with the other rows zeroed times B_id^T (R a multiple of 8,
    // steps of 16, the rest zero). A row meets only its own adapter, so all
    // adapters share one accumulator, which the row's factor then scales.
    const int R = g.ad.R;
    int id = lane < min(WR, rw) ? g.ad.ids[mw + lane] : -1;
    if (id < 0 || id >= g.ad.L) id = -1;
    const unsigned long long any = __ballot(id >= 0);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int col = tn * BN + wn * WC + j * 32 + (lane & 31);
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        float16v extra;
#pragma unroll
        for (int r = 0; r < 16; ++r) extra[r] = 0.0f;
        unsigned band = (unsigned)(any >> (32 * i));
        const int row = i * 32 + (lane & 31);
        while (band) {
          const int cur = __builtin_amdgcn_readlane(id, 32 * i + __builtin_ctz(band));
          const unsigned same = (unsigned)(__ballot(id == cur) >> (32 * i));
          band &= ~same;
          const bool mine = (same >> (lane & 31)) & 1u;
          const _Float16* bp =
              reinterpret_cast<const _Float16*>(g.ad.B) + ((size_t)cur * g.ncols + col) * R;
          const _Float16* tp = g.t16 + (size_t)(mw + row) * R;
          for (int k0 = 0; k0 < R; k0 += 16) {
            const int r0 = k0 + 8 * (lane >> 5);
            half8 a = {0, 0, 0, 0, 0, 0, 0, 0}, b = a;
            if (mine && r0 < R) a = *reinterpret_cast<const half8*>(tp + r0);
            if (col < g.ncols && r0 < R) b = *reinterpret_cast<const half8*>(bp + r0);
            extra = __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, extra, 0, 0, 0);
          }
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int m = mw + row_of(i, r);
          if (row_of(i, r) < rw && col < g.ncols)
            g.H[(size_t)m * g.ncols + col] =
                (_Float16)__builtin_fmaf(extra[r], g.ts[m], acc[i][j][r]);
        }
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int col = tn * BN + wn * WC + j * 32 + (lane & 31);
      if (col >= g.ncols) continue;
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          if (row_of(i, r) >= rw) continue;
          const int m = mw + row_of(i, r);
          const float v = acc[i][j][r] * g.rs[m];
          const uint32_t u = __builtin_bit_cast(uint32_t, v);
          g.dX[(size_t)m * g.ncols + col] =
              (u & 0x7fffffffu) > 0x7f800000u
                  ? (uint16_t)((u >> 16) | 0x40u)
                  : (uint16_t)((u + 0x7fffu + ((u >> 16) & 1u)) >> 16);
        }
    }
  }
}

// Tiles and splits of C[M][...]: 64-row tiles (56 KB of LDS, two workgroups a
// CU) up to 128 rows, 256-row tiles above; the contraction is split until the
// grid has one workgroup for every place on the GPU, in pieces of at least
// four steps.
void plan_tiles(FfnPlan& p, int M, int tiles_n, int nk) {
  p.BM = M <= 128 ? 64 : 256;
  p.tiles_m = (M + p.BM - 1) / p.BM;
  p.tiles_n = tiles_n;
  p.nk = nk;
  const long long tiles = (long long)p.tiles_m * tiles_n;
  const int places = p.BM == 64 ? 512 : 256;
  long long s = places / tiles;
  if (s > nk / 4) s = nk / 4;
  if (s < 1) s = 1;
  p.kper = (int)((nk + s - 1) / s);
  p.S = (nk + p.kper - 1) / p.kper;
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

template <Side SIDE>
hipError_t launch_tiles(TileArgs& g, const FfnPlan& p, hipStream_t st) {
  g.tiles_n = p.tiles_n;
  g.S = p.S;
  g.kper = p.kper;
  g.nk = p.nk;
  const long long grid = (long long)p.tiles_m * p.tiles_n * p.S;
  if (grid > 0x7fffffLL) return hipErrorInvalidValue;  // 2^32 lanes
  if (p.BM == 64)
    hipLaunchKernelGGL((ffn_gemm_kernel<64, SIDE>), dim3((unsigned)grid), dim3(2 * kRole), 0, st,
                       g);
  else
    hipLaunchKernelGGL((ffn_gemm_kernel<256, SIDE>), dim3((unsigned)grid), dim3(2 * kRole), 0,
                       st, g);
  return hipGetLastError();
}

}  // namespace

FfnPlan plan_glu_gemm(int M, int N, int K) {
  FfnPlan p{};
  plan_tiles(p, M, (N + 63) / 64, K / BK);
  p.ws_bytes = p.S > 1 ? (size_t)2 * p.S * M * N * sizeof(float) : 0;
  return p;
}

hipError_t launch_glu_gemm(const uint16_t* X, const uint8_t* Wg, const uint8_t* Wu, uint16_t* H,
                           uint16_t* G, uint16_t* U, int M, int N, int K, int act, void* ws,
                           const FfnPlan& p, hipStream_t st) {
  TileArgs g{};
  g.X = X;
  g.W0 = Wg;
  g.W1 = Wu;
  g.M = M;
  g.ncols = N;
  g.lda = K;
  g.NB = N / kBlockWeights;
  g.wrows = K;
  g.part = static_cast<float*>(ws);
  g.H = reinterpret_cast<_Float16*>(H);
  g.G = reinterpret_cast<_Float16*>(G);
  g.U = reinterpret_cast<_Float16*>(U);
  g.act = act;
  const hipError_t err = launch_tiles<kDual>(g, p, st);
  if (err != hipSuccess || p.S == 1) return err;
  return launch_glu_finish_f16(g.part, H, G, U, (size_t)M * N, p.S, act, st);
}

// Up to so many rows most use different adapters (requests that decode), and
// the narrow product is formed row by row.
constexpr int kFewRows = 64;

FfnPlan plan_gemm_lora(int M, int N, int K, int R) {
  FfnPlan p{};
  plan_tiles(p, M, (N + BN - 1) / BN, K / BK);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at = align256(at + bytes);
    return o;
  };
  if (M > kFewRows || p.S == 1) p.off_tp = take((size_t)shrink_shares(M, K) * M * R * sizeof(float));
  if (p.S > 1) {
    p.off_part = take((size_t)p.S * M * N * sizeof(float));
    p.off_t = take((size_t)M * R * sizeof(float));
  } else {
    p.off_t16 = take((size_t)M * R * 2);
    p.off_ts = take((size_t)M * sizeof(float));
  }
  p.ws_bytes = at;
  return p;
}

hipError_t launch_gemm_lora(const uint16_t* X, const uint8_t* B, const Adapters& ad, uint16_t* Y,
                            int M, int N, int K, void* ws, const FfnPlan& p, hipStream_t st) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  float* t = p.S > 1 ? reinterpret_cast<float*>(w + p.off_t) : nullptr;
  uint16_t* t16 = p.S > 1 ? nullptr : reinterpret_cast<uint16_t*>(w + p.off_t16);
  float* ts = p.S > 1 ? nullptr : reinterpret_cast<float*>(w + p.off_ts);
  float* tp = M > kFewRows || p.S == 1 ? reinterpret_cast<float*>(w + p.off_tp) : nullptr;
  hipError_t err = launch_lora_shrink_f16(X, ad, tp, t, t16, ts, M, K, st);
  if (err != hipSuccess) return err;
  TileArgs g{};
  g.X = X;
  g.W0 = B;
  g.M = M;
  g.ncols = N;
  g.lda = K;
  g.NB = N / kBlockWeights;
  g.wrows = K;
  g.part = reinterpret_cast<float*>(w + p.off_part);
  g.H = reinterpret_cast<_Float16*>(Y);
  g.t16 = reinterpret_cast<const _Float16*>(t16);
  g.ts = ts;
  g.ad = ad;
  err = launch_tiles<kAdapters>(g, p, st);
  if (err != hipSuccess || p.S == 1) return err;
  return launch_lora_finish_f16(g.part, t, ad, Y, M, N, p.S, st);
}

FfnPlan plan_gradient(int M, int N, int K, int mats) {
  FfnPlan p{};
  plan_tiles(p, M, (K + BN - 1) / BN, mats * (N / BK));
  p.off_a = 0;
  size_t at = align256((size_t)M * mats * N * 2);
  p.off_rs = at;
  at = align256(at + (size_t)M * sizeof(float));
  p.off_part = at;
  if (p.S > 1) at += (size_t)p.S * M * K * sizeof(float);
  p.ws_bytes = at;
  return p;
}

hipError_t launch_gradient(const uint16_t* dH, const uint16_t* G, const uint16_t* U,
                           const uint8_t* W0, const uint8_t* W1, uint16_t* dX, int M, int N, int K,
                           int act, int mats, void* ws, const FfnPlan& p, hipStream_t st) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  uint16_t* a = reinterpret_cast<uint16_t*>(w + p.off_a);
  float* rs = reinterpret_cast<float*>(w + p.off_rs);
  hipError_t err = launch_gradient_rows(dH, G, U, a, rs, M, N, act, mats, st);
  if (err != hipSuccess) return err;
  TileArgs g{};
  g.X = a;
  g.W0 = W0;
  g.W1 = W1;
  g.M = M;
  g.ncols = K;
  g.lda = mats * N;
  g.NB = N / kBlockWeights;
  g.wrows = K;
  g.nk_mat = N / BK;
  g.part = reinterpret_cast<float*>(w + p.off_part);
  g.dX = dX;
  g.rs = rs;
  err = launch_tiles<kGradient>(g, p, st);
  if (err != hipSuccess || p.S == 1) return err;
  return launch_gradient_finish(g.part, rs, dX, M, K, p.S, st);
}

}  // namespace q4
