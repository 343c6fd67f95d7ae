// Prompt and gradient GEMMs of the dense feed-forward operators over Q4_0
// weights, on the fp16 matrix cores with fp32 sums:
//   dual      H = act(X . deq(Wg)) * (X . deq(Wu))            X fp16 [M][K]
//   adapters  Y = X . deq(B) + t . B_id^T                     X fp16 [M][K]
//   gradient  dX = dG . deq(Wg)^T + dU . deq(Wu)^T            one or two matrices
//
// Tile BM x 128, K steps of 64. Consumer waves issue the matrix instructions, 4
// producer waves fetch the weights and dequantize them into an fp16 LDS tile
// [column][k], so the VALU work of one role runs beside the matrix work of the
// other. LDS holds two steps; a barrier a step hands over. Up to 128 rows there are
// 4 consumer waves and the producers copy the left operand too. At 256 rows there
// are 8, two a SIMD, which copy it themselves: with 4 and 4 waves both roles had
// 2000 cycles of a step's 2270 to do (777 rows of 5120 x 1536, gradient: 49.5 us;
// 8 consumers 46.5, and copying 45.6; 2048 rows of 4096 x 4096: 77.3, 75.4, 74.5).
//
//   * Left operand: 16-byte loads into registers, two steps ahead, and 16-byte
//     LDS stores, XOR-swizzled.
//   * Weights: a producer lane loads a block of a step straight into registers,
//     two steps ahead, and writes the dequantized values one step ahead. The raw
//     bytes never pass through LDS.
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
// Each dequantized weight w = (q - 8) * d is rounded to fp16 before its product,
// as in q4_0_gemm; the sums are fp32. Rounded weights give g and u an error of
// about 0.8 of what rounding them to fp16 gives, and h, their product, one 1.5
// times that of its own rounding. So dual adds the products of what the rounding
// took, for all weights: w - fp16(w) is at most 4 of d's last places, which an 8-bit
// float (fp16's exponents, 2 bits of mantissa) holds exactly, and 8-bit products run
// at twice fp16's rate, 64 of k an instruction. There x is cut to its upper byte, off
// by less than a quarter and by a tenth on the whole, so that of the roundings at
// most a quarter is left: 1.006 times. 2048 rows of 4096 x 11008: 503 us, without
// these products 397, with fp16 ones 800 (1.000 times). The adapters' projection
// rounds its weights and no more, as q4_0_gemm does: its result is one product, off by
// 1.24 to 1.29 times its own rounding; with the roundings' products 1.003 to 1.03, but
// 262 against 209 us at 2000 rows of 11008 x 4096. The gradients have bf16 results,
// eight times coarser, and round the weights.
//
// What bounds it: a step of 256 rows is 1024 cycles of matrix instructions (dual
// 1536) and moves 176 KiB through LDS (dual 216). With all CUs busy the power limit
// holds the clock at 1.6 to 1.75 GHz, and moving work between the roles gives 2 to
// 4 %; with 160 CUs busy the clock is 2.4 GHz and the producers' chain is the long one
// (their weights; consumers wait 500 to 900 of 2700 cycles). Raised wave priorities and
// deeper prefetch gave nothing.
#include <algorithm>
#include <type_traits>

#include "ffn_device.hpp"
#include "ffn_internal.hpp"
#include "q4_device.hpp"

namespace q4 {
namespace {

typedef float float16v __attribute__((ext_vector_type(16)));
typedef int int8v __attribute__((ext_vector_type(8)));

constexpr int BN = 128, BK = 64;
constexpr int kRole = 256;                 // lanes of one role
constexpr int kColBytes = BK * 2;          // one column or row of a step in LDS
constexpr int kBBytes = BN * kColBytes;    // 16 KiB
constexpr uint32_t kOut = 0x80000000u;    // past the end of any weight matrix

enum Side { kAdapters, kDual, kGradient };

// dual: the roundings of a step's weights as 8-bit floats, beside the weights.
template <Side SIDE>
constexpr bool kRest = SIDE == kDual;
template <Side SIDE>
constexpr int kWeightBytes = kBBytes + (kRest<SIDE> ? BN * BK : 0);  // of a step, in LDS

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

// Roundings in LDS: column n's 64 bytes are four pieces of 16, piece 2 * h + p those
// of quarters 2p and 2p + 1 of the step that lane half h multiplies. Four columns
// share a line of 256 bytes, in which the pieces are permuted by the column's bits
// 2, 3, 4 and 6, so that neither the 16 columns of a read nor the 8 of a store meet
// in a bank.
__device__ __forceinline__ int rest_piece(int n, int piece) {
  const int swz = ((n >> 3) & 1) | ((n >> 2) & 1) << 1 | ((n >> 4) & 1) << 2 | ((n >> 6) & 1) << 3;
  return (n >> 2) * 256 + ((((n & 3) * 4 + piece) ^ swz) << 4);
}

__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Hands LDS over at a barrier: this wave's reads and writes of it are done before
// the barrier. Neither the wait nor the barrier is an access of memory to the
// compiler, so both orders are stated: none of them may be moved past the wait, in
// the program (memory clobber) or among the instructions (scheduling barrier).
__device__ __forceinline__ void lds_hand_over() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
  lds_barrier();
}

// Nibbles to scaled halves, two at a time. binary16 0x6400 | v is 1024 + v
// exactly, and 0x5400 | (v << 4) is 64 + v, so every other nibble needs no
// shift; (q - 8) is exact, the product is rounded once. The masks are kept in
// vector registers, so that masking and setting the exponent is one instruction
// (which takes at most one constant from elsewhere).
struct Dequant {
  uint32_t even = 0x000f000fu, odd = 0x00f000f0u;
  __device__ __forceinline__ Dequant() { asm volatile("" : "+v"(even), "+v"(odd)); }
  // q - 8 of the nibbles at bits 0 and 16, or 4 and 20
  __device__ __forceinline__ half2v low_value(uint32_t q) const {
    const half2v off = {(_Float16)1032.0f, (_Float16)1032.0f};
    return __builtin_bit_cast(half2v, (q & even) | 0x64006400u) - off;
  }
  __device__ __forceinline__ half2v high_value(uint32_t q) const {
    const half2v off = {(_Float16)72.0f, (_Float16)72.0f};
    return __builtin_bit_cast(half2v, (q & odd) | 0x54005400u) - off;
  }
  __device__ __forceinline__ uint32_t low(uint32_t q, half2v d) const {
    return __builtin_bit_cast(uint32_t, low_value(q) * d);
  }
  __device__ __forceinline__ uint32_t high(uint32_t q, half2v d) const {
    return __builtin_bit_cast(uint32_t, high_value(q) * d);
  }
  // What the rounding of w = v * d took, times 2^8: v * d - w is a whole number of at
  // most 4 of d's last places, which fp16 holds, and times 2^8 its upper byte alone
  // does, as an 8-bit float of fp16's exponents (for every d and nibble whose w is
  // finite).
  static __device__ __forceinline__ uint32_t rest(half2v v, half2v d, half2v w) {
    const half2v r = __builtin_elementwise_fma(v, d, -w);
    const half2v s = {(_Float16)256.0f, (_Float16)256.0f};
    return __builtin_bit_cast(uint32_t, r * s);
  }
};

// The upper bytes of four halves: truncated to two bits of mantissa, as 8-bit floats
// of the same exponents.
__device__ __forceinline__ uint32_t upper_bytes(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x07050301u);
}

// ---------------------------------------------------------------- weights
// Two registers of a lane pair 32 (16) lanes apart: afterwards a holds the lower
// lane's values and b the upper lane's, of register a in the lower lane and of
// register b in the upper one.
__device__ __forceinline__ void swap32(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}
__device__ __forceinline__ void swap16(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}

// Forward: the step's 64 weight rows x 4 blocks are one block a producer lane,
// two loads. Wave w takes rows 32 * (w % 2) .. of
// the column half w / 2 (dual: half 0 is the gate, half 1 the up matrix); in the
// row number of lane l bit 0 is l / 32, bit 1 is l / 16 % 2, the rest l / 2 % 8;
// its block is l % 2. The four lanes that hold one block column of four
// consecutive rows exchange dwords by lane swaps (a 4 x 4 transposition), which
// leaves each with dword 2 * (l / 32) + l / 16 % 2 of all four rows: 4 rows x 8
// columns.
template <bool DUAL>
struct ForwardWeights {
  __amdgpu_buffer_rsrc_t r;
  Dequant dq;
  uint32_t vq, vd, pitch;
  int n0, chunk, half;
  int rest_at;  // place of the roundings in column n0
  struct Raw {
    uint32_t q[4], d;
  };
  __device__ __forceinline__ void init(const TileArgs& g, int tn, int t) {
    const int w = __builtin_amdgcn_readfirstlane(t >> 6);
    const int l = t & 63;
    const int hw = w >> 1;
    const int blk = l & 1, b4 = (l >> 4) & 1, b5 = l >> 5;
    const int rg = 8 * (w & 1) + ((l >> 1) & 7);
    pitch = (uint32_t)g.NB * kBlockBytes;
    const uint8_t* base = (DUAL && hw) ? g.W1 : g.W0;
    r = make_rsrc(base, (uint32_t)g.wrows * pitch);
    const int col = DUAL ? 2 * tn + blk : 4 * tn + 2 * hw + blk;  // block column
    // a block column past the matrix reads zeros
    const uint32_t o = (uint32_t)(4 * rg + 2 * b4 + b5) * pitch + (uint32_t)col * kBlockBytes;
    vd = col < g.NB ? o : kOut;
    vq = col < g.NB ? o + 2 : kOut;
    n0 = (DUAL ? 2 * blk + hw : 2 * hw + blk) * 32 + (2 * b5 + b4) * 8;
    chunk = rg >> 1;
    half = rg & 1;
    // row 4 * rg is k = 16 * (rg / 4) + 4 * (rg % 4)
    rest_at = rest_piece(n0, (rg & 2) + (rg >> 3)) + 8 * ((rg >> 2) & 1) + 4 * (rg & 1);
  }
  // all loads go with part 0
  __device__ __forceinline__ void load(Raw& raw, int ks, int i) const {
    if (i != 0) return;
    const uint32_t so = (uint32_t)ks * (BK * pitch);
    const auto v = __builtin_amdgcn_raw_buffer_load_b128(r, vq, so, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) raw.q[j] = v[j];
    raw.d = __builtin_amdgcn_raw_buffer_load_b16(r, vd, so, 0);
  }
  // a unit taken out of its registers: row pairs side by side, columns 0..3 from
  // the low halves of the rows' dwords, 4..7 from the high ones
  struct Taken {
    uint32_t p01[2], p23[2];
    half2v d01, d23;
  };
  __device__ __forceinline__ void take(const Raw& raw, Taken& k) const {
    uint32_t q0 = raw.q[0], q1 = raw.q[1], q2 = raw.q[2], q3 = raw.q[3];
    swap32(q0, q2);
    swap32(q1, q3);
    swap16(q0, q1);
    swap16(q2, q3);  // rows 0, 2, 1, 3
    uint32_t da = raw.d, db = raw.d;
    swap32(da, db);
    uint32_t p = (da & 0xffffu) | (db << 16), p2 = p;
    swap16(p, p2);
    k.d01 = __builtin_bit_cast(half2v, p);
    k.d23 = __builtin_bit_cast(half2v, p2);
    k.p01[0] = __builtin_amdgcn_perm(q2, q0, 0x05040100u);
    k.p01[1] = __builtin_amdgcn_perm(q2, q0, 0x07060302u);
    k.p23[0] = __builtin_amdgcn_perm(q3, q1, 0x05040100u);
    k.p23[1] = __builtin_amdgcn_perm(q3, q1, 0x07060302u);
  }
  // columns 2 * part and 2 * part + 1
  __device__ __forceinline__ void store(const Taken& k, uint8_t* __restrict__ bs, int part) const {
    const int sh = 8 * (part & 1);
    const uint32_t a = k.p01[part >> 1] >> sh, b = k.p23[part >> 1] >> sh;
    store_column(bs, 2 * part, dq.low_value(a), dq.low_value(b), k);
    store_column(bs, 2 * part + 1, dq.high_value(a), dq.high_value(b), k);
  }
  __device__ __forceinline__ void store_column(uint8_t* __restrict__ bs, int c, half2v v01,
                                               half2v v23, const Taken& k) const {
    const int n = n0 + c;
    const half2v w01 = v01 * k.d01, w23 = v23 * k.d23;
    *reinterpret_cast<uint2*>(bs + n * kColBytes + ((chunk ^ swz_b(n)) << 4) + half * 8) =
        make_uint2(__builtin_bit_cast(uint32_t, w01), __builtin_bit_cast(uint32_t, w23));
    if constexpr (DUAL)
      // rest_piece(n0 + c, ..): n0 is a multiple of 8
      *reinterpret_cast<uint32_t*>(bs + kBBytes + (c >> 2) * 256 +
                                   (rest_at ^ (((c & 3) * 4 ^ (c >> 2) * 2) << 4))) =
          upper_bytes(Dequant::rest(v01, k.d01, w01), Dequant::rest(v23, k.d23, w23));
  }
};

// Gradient: the step's tile is 128 weight rows x 2 blocks, one block a
// producer lane (row t / 2, block t % 2).
struct GradientWeights {
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
  // all loads go with part 3, when the registers are free
  __device__ __forceinline__ void load(Raw& raw, int ks, int i) const {
    if (i != 3) return;
    const bool second = ks >= nk_mat;
    const uint32_t so = (uint32_t)(second ? ks - nk_mat : ks) * (2 * kBlockBytes);
    const __amdgpu_buffer_rsrc_t r = second ? r1 : r0;
    const auto v = __builtin_amdgcn_raw_buffer_load_b128(r, vq, so, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) raw.q[j] = v[j];
    raw.d = __builtin_amdgcn_raw_buffer_load_b16(r, vd, so, 0);
  }
  struct Taken {
    uint32_t q[4];
    half2v d;
  };
  __device__ __forceinline__ void take(const Raw& raw, Taken& k) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) k.q[j] = raw.q[j];
    k.d = __builtin_bit_cast(half2v, (raw.d & 0xffffu) | (raw.d << 16));
  }
  // dword `part` of the block
  __device__ __forceinline__ void store(const Taken& k, uint8_t* __restrict__ bs, int part) const {
    const uint32_t q = k.q[part], q8 = q >> 8;
    uint4 v;
    v.x = dq.low(q, k.d);
    v.y = dq.high(q, k.d);
    v.z = dq.low(q8, k.d);
    v.w = dq.high(q8, k.d);
    *reinterpret_cast<uint4*>(bs + n * kColBytes + (((4 * b + part) ^ swz_b(n)) << 4)) = v;
  }
};

// Consumer waves. Eight, two a SIMD, have time to copy the left operand as well.
template <int BM>
constexpr int kConsumers = BM == 256 ? 8 : 4;
template <int BM>
constexpr bool kConsumersCopy = BM == 256;
template <int BM>
constexpr int kTileThreads = kConsumers<BM> * kWaveSize + kRole;

// ---------------------------------------------------------------- left operand
// A step's left operand through registers: 16-byte loads, 16-byte LDS stores.
// (LDS-DMA copies of 16 bytes a lane kept the address unit busy for 60 to 80
// cycles each, 32 of them a step of 256 rows.)
template <int BM, int LANES>
struct LeftOperand {
  static constexpr int kInstr = BM * kColBytes / 16 / LANES;
  __amdgpu_buffer_rsrc_t r;
  uint32_t off[kInstr];
  int t;
  struct Raw {
    uint4 v[kInstr];
  };
  __device__ __forceinline__ void init(const TileArgs& g, int m0, int rows, int lane) {
    t = lane;
    const uint32_t pitch = (uint32_t)g.lda * 2u, bytes = (uint32_t)rows * pitch;
    r = make_rsrc(g.X + (size_t)m0 * g.lda, bytes);
    // Rows past the last read zeros, not kept; where 256 rows of a contraction of 2N
    // pass 2 GiB, kOut is inside, and they repeat the last row. (Repeating it always:
    // 150 rows of 11008 x 4096 35.3 -> 36.0 us.)
    const uint32_t dead = bytes <= kOut ? kOut : bytes - pitch;
#pragma unroll
    for (int i = 0; i < kInstr; ++i) {
      const int slot = i * LANES + t;  // row slot / 8, 16-byte chunk slot % 8
      const int row = slot >> 3;
      off[i] = (row < rows ? (uint32_t)row * pitch : dead) + 16u * (slot & 7);
    }
  }
  __device__ __forceinline__ void load(Raw& raw, int ks, int i) const {
    const auto v = __builtin_amdgcn_raw_buffer_load_b128(r, off[i], (uint32_t)ks * kColBytes, 0);
    raw.v[i] = make_uint4(v[0], v[1], v[2], v[3]);
  }
  __device__ __forceinline__ void store(const Raw& raw, uint8_t* __restrict__ stage, int i) const {
    const int slot = i * LANES + t;
    const int row = slot >> 3;
    *reinterpret_cast<uint4*>(stage + row * kColBytes + (((slot & 7) ^ swz_x(row)) << 4)) =
        raw.v[i];
  }
};

// How many steps ahead the producers load, into registers. Few rows leave little
// to do in a step, so that more of them have to be in flight.
template <int BM>
constexpr int kDepth = BM == 64 ? 4 : 2;

// What the producers do while step ks is multiplied: store ks + 1 from its
// registers into its LDS tiles, dequantized, and load ks + 1 + D into them (the left
// operand where the consumers do not copy it). Steps
// past the last repeat it, into registers that are not read.
template <int BM, class W>
__device__ __forceinline__ void produce_step(const W& wt, const LeftOperand<BM, kRole>& left,
                                             typename W::Raw& raw,
                                             typename LeftOperand<BM, kRole>::Raw& lraw,
                                             uint8_t* __restrict__ x, uint8_t* __restrict__ b,
                                             int next) {
  typename W::Taken k;
  wt.take(raw, k);
  constexpr int kInstr = kConsumersCopy<BM> ? 0 : LeftOperand<BM, kRole>::kInstr;
  constexpr int kPer = (kInstr + 3) / 4;
#pragma unroll
  for (int part = 0; part < 4; ++part) {
    wt.store(k, b, part);
    wt.load(raw, next, part);
#pragma unroll
    for (int i = part * kPer; i < part * kPer + kPer; ++i)
      if (i < kInstr) {
        left.store(lraw, x, i);
        left.load(lraw, next, i);
      }
    __builtin_amdgcn_sched_barrier(0);
  }
  lds_hand_over();
}

// The producer waves (lane t of them) over the K steps [kb, ke).
template <int BM, Side SIDE>
__device__ __forceinline__ void produce(const TileArgs& g, uint8_t* __restrict__ xs,
                                        uint8_t* __restrict__ bs, int m0, int rows, int tn, int kb,
                                        int ke, int t) {
  using W = typename std::conditional<SIDE == kGradient, GradientWeights,
                                      ForwardWeights<SIDE == kDual>>::type;
  constexpr int D = kDepth<BM>;
  constexpr int kXBytes = BM * kColBytes;
  constexpr int kStage = kWeightBytes<SIDE>;
  W wt;
  wt.init(g, tn, t);
  LeftOperand<BM, kRole> left;
  if constexpr (!kConsumersCopy<BM>) left.init(g, m0, rows, t);
  typename W::Raw raw[D];
  typename LeftOperand<BM, kRole>::Raw lraw[D];
#pragma unroll
  for (int d = 0; d < D; ++d) {
#pragma unroll
    for (int part = 0; part < 4; ++part) wt.load(raw[d], min(kb + d, ke - 1), part);
#pragma unroll
    for (int i = 0; i < LeftOperand<BM, kRole>::kInstr; ++i)
      if constexpr (!kConsumersCopy<BM>) left.load(lraw[d], min(kb + d, ke - 1), i);
    __builtin_amdgcn_sched_barrier(0);
  }
  produce_step<BM>(wt, left, raw[0], lraw[0], xs, bs, min(kb + D, ke - 1));
  // unrolled so that registers and LDS tiles are named at compile time
  static_assert(D % 2 == 0, "the LDS tiles alternate");
  int ks = kb;
  for (; ks + D <= ke; ks += D) {
#pragma unroll
    for (int u = 0; u < D; ++u)
      produce_step<BM>(wt, left, raw[(u + 1) % D], lraw[(u + 1) % D],
                       xs + ((u + 1) & 1) * kXBytes, bs + ((u + 1) & 1) * kStage,
                       min(ks + u + 1 + D, ke - 1));
  }
#pragma unroll
  for (int u = 0; u < D - 1; ++u)
    if (ks + u < ke)
      produce_step<BM>(wt, left, raw[(u + 1) % D], lraw[(u + 1) % D],
                       xs + ((u + 1) & 1) * kXBytes, bs + ((u + 1) & 1) * kStage, ke - 1);
}

template <int BM, Side SIDE>
__global__ __launch_bounds__(kTileThreads<BM>, BM == 256 ? 3 : 4) void ffn_gemm_kernel(TileArgs g) {
  constexpr int kXBytes = BM * kColBytes;
  constexpr int kStage = kWeightBytes<SIDE>;
  // two steps' left operand and weights; at the end the waves' results
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * kXBytes + 2 * kStage];
  uint8_t* xs = lds;
  uint8_t* bs = lds + 2 * kXBytes;
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

  constexpr int NC = kConsumers<BM>;
  if (wave >= NC) {
    produce<BM, SIDE>(g, xs, bs, m0, rows, tn, kb, ke, (int)threadIdx.x - NC * kWaveSize);
    return;
  }

  // -------------------------------------------------------------- consumer
  const int lane = threadIdx.x & 63;
  constexpr int WGR = BM == 256 ? 4 : 2;  // waves along the rows
  constexpr int WR = BM / WGR;            // rows of a wave: 64 or 32
  constexpr int WC = BN / (NC / WGR);     // columns of a wave: 64
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
  // A quarter of a step (16 of k) at a time: its operands, then its products.
  constexpr bool REST = kRest<SIDE>;
  struct Operands {
    half8 a[MI], b[NJ];
  };
  const int ra = wm * WR + (lane & 31), rb = wn * WC + (lane & 31);
  // A lane's place in the stages in quarter 0; quarter kk is 2 * kk chunks on, before
  // the swizzle, the next 32 rows swizzled alike, the next 32 columns by one more.
  int xo = ra * kColBytes + (((lane >> 5) ^ swz_x(ra)) << 4);
  int bo = rb * kColBytes + (((lane >> 5) ^ swz_b(rb)) << 4);
  auto read = [&](Operands& o, const uint8_t* x, const uint8_t* b, int kk) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
      o.a[i] = *reinterpret_cast<const half8*>(x + (xo ^ (kk << 5)) + 32 * i * kColBytes);
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      o.b[j] =
          *reinterpret_cast<const half8*>(b + (bo ^ (kk << 5) ^ (j << 4)) + 32 * j * kColBytes);
  };
  auto multiply = [&](const Operands& o) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(o.b[j], o.a[i], acc[i][j], 0, 0, 0);
  };
  // The roundings' products, a whole step's (64 of k) at once in 8-bit floats. The
  // lane's 32 values of k are those of its four quarters, on both sides.
  struct Rest {
    int8v b[REST ? NJ : 1], a[REST ? MI : 1];
  };
  int ro = kBBytes + rest_piece(rb, 2 * (lane >> 5));
  auto read_rest = [&](Rest& t, const uint8_t* b) {
#pragma unroll
    for (int j = 0; j < NJ; ++j)  // 32 columns on are 8 lines
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const uint4 v = *reinterpret_cast<const uint4*>(b + (ro ^ (p << 4)) + 32 * BK * j);
        t.b[j][4 * p] = v.x, t.b[j][4 * p + 1] = v.y, t.b[j][4 * p + 2] = v.z,
                  t.b[j][4 * p + 3] = v.w;
      }
  };
  auto take_rest = [&](Rest& t, const Operands& o, int q) {  // the left operand of quarter q
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const uint4 v = __builtin_bit_cast(uint4, o.a[i]);
      t.a[i][2 * q] = upper_bytes(v.x, v.y);
      t.a[i][2 * q + 1] = upper_bytes(v.z, v.w);
    }
  };
  auto multiply_rest = [&](const Rest& t) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j)  // scales 2^-8 and 1, formats 5 exponent bits and 2 more
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
            t.b[j], t.a[i], acc[i][j], 1, 1, 0, 0x77777777, 0, 0x7f7f7f7f);
  };
  // One or two consumer waves a SIMD: little else hides the latency of their LDS
  // reads, so the reads of a quarter are issued before the products of the one
  // before, and a step's last products run after the barrier, over the first reads
  // of the next step.
  constexpr int Q = BK / 16;
  constexpr bool COPY = kConsumersCopy<BM>;
  using Left = LeftOperand<BM, NC * kWaveSize>;
  Left left;
  constexpr int SETS = REST ? 1 : 2;  // steps of it in flight: registers are short beside roundings
  typename Left::Raw lraw[SETS];
  if constexpr (COPY) {
    left.init(g, m0, rows, (int)threadIdx.x);
#pragma unroll
    for (int d = 0; d < SETS; ++d)
#pragma unroll
      for (int i = 0; i < Left::kInstr; ++i) left.load(lraw[d], min(kb + d, ke - 1), i);
#pragma unroll
    for (int i = 0; i < Left::kInstr; ++i) {
      left.store(lraw[0], xs, i);
      left.load(lraw[0], min(kb + SETS, ke - 1), i);
    }
  }
  lds_hand_over();
  if constexpr (MI * NJ <= 2) {
    // few products: all of a step's reads at once
    Operands o[Q];
    for (int ks = kb; ks < ke; ++ks) {
      const int cur = (ks - kb) & 1;
      const uint8_t* x = xs + cur * kXBytes;
      const uint8_t* b = bs + cur * kStage;
#pragma unroll
      for (int q = 0; q < Q; ++q) read(o[q], x, b, q);
      Rest rest;
      if constexpr (REST) read_rest(rest, b);
      lds_hand_over();  // this wave's reads done before the stages are reused
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        if constexpr (REST) take_rest(rest, o[q], q);
        multiply(o[q]);
      }
      if constexpr (REST) multiply_rest(rest);
    }
  } else {
    Operands o[2];
    read(o[0], xs, bs, 0);
    auto step = [&](int ks, typename Left::Raw& next) __attribute__((always_inline)) {
      const int cur = (ks - kb) & 1;
      const uint8_t* x = xs + cur * kXBytes;
      const uint8_t* b = bs + cur * kStage;
      // beside roundings formed anew in each step: kept, the quarters' addresses take 12 registers
      if constexpr (REST) asm volatile("" : "+v"(xo), "+v"(bo), "+v"(ro));
      Rest rest;
#pragma unroll
      for (int q = 0; q < Q - 1; ++q) {
        read(o[(q + 1) & 1], x, b, q + 1);
        if constexpr (COPY) {
          constexpr int kPer = (Left::kInstr + Q - 2) / (Q - 1);
#pragma unroll
          for (int i = q * kPer; i < q * kPer + kPer; ++i)
            if (i < Left::kInstr) {
              left.store(next, xs + (cur ^ 1) * kXBytes, i);
              left.load(next, min(ks + 1 + SETS, ke - 1), i);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (REST) take_rest(rest, o[q & 1], q);
        multiply(o[q & 1]);
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (REST) {  // the roundings' products are the step's last
        read_rest(rest, b);
        __builtin_amdgcn_sched_barrier(0);
        take_rest(rest, o[(Q - 1) & 1], Q - 1);
        multiply(o[(Q - 1) & 1]);
        __builtin_amdgcn_sched_barrier(0);
      }
      lds_hand_over();  // reads and copies done before the stages change roles
      __builtin_amdgcn_sched_barrier(0);
      // past the last step this reads a stage that is not used
      read(o[0], xs + (cur ^ 1) * kXBytes, bs + (cur ^ 1) * kStage, 0);
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (REST)
        multiply_rest(rest);
      else
        multiply(o[(Q - 1) & 1]);
      __builtin_amdgcn_sched_barrier(0);
    };
    if constexpr (COPY && SETS == 2) {  // the sets of registers are named at compile time
      int ks = kb;
      for (; ks + 2 <= ke; ks += 2) {
        step(ks, lraw[1]);
        step(ks + 1, lraw[0]);
      }
      if (ks < ke) step(ks, lraw[1]);
    } else {
      for (int ks = kb; ks < ke; ++ks) step(ks, lraw[0]);
    }
  }

  // The weights are the left operand of the instruction, so a 32 x 32 result has
  // its rows along the tile's columns: lane l holds row l % 32 of X, register r
  // column 8 * (r / 4) + 4 * (l / 32) + r % 4. Four registers are four
  // neighbouring columns.
  const int mw = m0 + wm * WR;    // first row of the wave
  const int rw = rows - wm * WR;  // its live rows
  const int lr = lane & 31, l4 = 4 * (lane >> 5);

  if (g.S > 1) {
    const size_t slab = (size_t)g.M * g.ncols;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int v = wn * WC + j * 32;  // column of the tile
      const int mat = SIDE == kDual ? (v >> 5) & 1 : 0;
      const int col = (SIDE == kDual ? tn * 64 + (v >> 6) * 32 : tn * BN + v) + l4;
      if (col >= g.ncols) continue;  // 32 columns of a tile are all inside or all outside
      float* dst = g.part + ((size_t)mat * g.S + sp) * slab + col;
#pragma unroll
      for (int i = 0; i < MI; ++i)
        if (32 * i + lr < rw)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<float4*>(dst + (size_t)(mw + 32 * i + lr) * g.ncols + 8 * q) =
                make_float4(acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                            acc[i][j][4 * q + 3]);
    }
    return;
  }

  // Results go through the wave's own part of LDS and leave in whole 16-byte
  // pieces of rows (stored from the registers, two bytes a lane, the 256 x 64
  // block of three results took 20000 cycles, as long as nine K steps).
  constexpr int OC = SIDE == kDual ? WC / 2 : WC;  // result columns of the wave
  constexpr int kPitch = OC * 2 + 16;              // bytes of an LDS row
  static_assert(NC * WR * kPitch <= 2 * kXBytes + 2 * kStage, "results fit the stages");
  uint8_t* out = lds + wave * (WR * kPitch);
  const int col0 = SIDE == kDual ? tn * 64 + wn * OC : tn * BN + wn * OC;
  auto put = [&](int i, int j, const uint2(&v)[4]) {  // 32 rows x 32 columns
#pragma unroll
    for (int q = 0; q < 4; ++q)
      *reinterpret_cast<uint2*>(out + (32 * i + lr) * kPitch + (32 * j + 8 * q + l4) * 2) = v[q];
  };
  auto flush = [&](uint16_t* dst) {
    constexpr int kPieces = OC / 8;  // 16-byte pieces of a row
#pragma unroll
    for (int o = 0; o < WR * kPieces; o += kWaveSize) {
      const int row = (o + lane) / kPieces, pc = (o + lane) % kPieces;
      if (row < rw && col0 + 8 * pc < g.ncols)
        *reinterpret_cast<uint4*>(dst + (size_t)(mw + row) * g.ncols + col0 + 8 * pc) =
            *reinterpret_cast<const uint4*>(out + row * kPitch + 16 * pc);
    }
  };
  auto pack16 = [](float a, float b, float c, float d) {
    typedef _Float16 half4 __attribute__((ext_vector_type(4)));
    return __builtin_bit_cast(uint2, half4{(_Float16)a, (_Float16)b, (_Float16)c, (_Float16)d});
  };

  if constexpr (SIDE == kDual) {
#pragma unroll
    for (int what = 0; what < 3; ++what) {  // g and u, then h (acc is formed last)
      if (what < 2 && !g.G) continue;
#pragma unroll
      for (int j = 0; j < NJ; j += 2)
#pragma unroll
        for (int i = 0; i < MI; ++i) {
          uint2 v[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float e[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const float gt = acc[i][j][4 * q + u], up = acc[i][j + 1][4 * q + u];
              e[u] = what == 0 ? gt : (what == 1 ? up : act_value<true>(gt, g.act) * up);
            }
            v[q] = pack16(e[0], e[1], e[2], e[3]);
          }
          put(i, j / 2, v);
        }
      flush(reinterpret_cast<uint16_t*>(what == 0 ? g.G : (what == 1 ? g.U : g.H)));
    }
  } else if constexpr (SIDE == kAdapters) {
    // Wide half of the adapters: for every adapter that occurs in the wave's
    // rows, t16 times B_id^T (R a multiple of 8, steps of 16, the rest zero),
    // which the adapter's own rows scale and add: an infinity or NaN in one
    // adapter stays with the rows that use it. The loads of all columns and of kC
    // steps go out together: with many adapters in a tile most of the time goes
    // by waiting for them.
    constexpr int kC = 2;
    const int R = g.ad.R;
    const int r8 = 8 * (lane >> 5);
    int id = lane < min(WR, rw) ? g.ad.ids[mw + lane] : -1;
    if (id < 0 || id >= g.ad.L) id = -1;
    const unsigned long long any = __ballot(id >= 0);
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int row = min(32 * i + lr, rw - 1);
      const float ts = g.ts[mw + row];
      const _Float16* tp = g.t16 + (size_t)(mw + row) * R;
      unsigned band = (unsigned)(any >> (32 * i));
      while (band) {
        const int cur = __builtin_amdgcn_readlane(id, 32 * i + __builtin_ctz(band));
        const unsigned same = (unsigned)(__ballot(id == cur) >> (32 * i));
        band &= ~same;
        const bool mine = (same >> lr) & 1u;
        const _Float16* bp = reinterpret_cast<const _Float16*>(g.ad.B) +
                             ((size_t)cur * g.ncols + min(col0, g.ncols - 32) + lr) * R;
        for (int k0 = 0; k0 < R; k0 += 16 * kC) {
          half8 a[kC], b[NJ][kC];
#pragma unroll
          for (int c = 0; c < kC; ++c) {
            const int at = k0 + 16 * c;
            if (at >= R) break;  // uniform
            // past R the left operand is zero and the right one some of the same
            // adapter's; columns past the matrix are not kept
            const int r0 = min(at + r8, R - 8);
            a[c] = *reinterpret_cast<const half8*>(tp + r0);
            if (at + r8 >= R) a[c] = half8{0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < NJ; ++j)
              b[j][c] = *reinterpret_cast<const half8*>(
                  bp + (uint32_t)((col0 + 32 * j < g.ncols ? 32 * j : 0) * R + r0));
          }
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            float16v own;
#pragma unroll
            for (int r = 0; r < 16; ++r) own[r] = 0.0f;
#pragma unroll
            for (int c = 0; c < kC; ++c)
              if (k0 + 16 * c < R)
                own = __builtin_amdgcn_mfma_f32_32x32x16_f16(b[j][c], a[c], own, 0, 0, 0);
#pragma unroll
            for (int r = 0; r < 16; ++r)
              acc[i][j][r] = mine ? __builtin_fmaf(own[r], ts, acc[i][j][r]) : acc[i][j][r];
          }
        }
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        uint2 v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          v[q] = pack16(acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                        acc[i][j][4 * q + 3]);
        put(i, j, v);
      }
    }
    flush(reinterpret_cast<uint16_t*>(g.H));
  } else {
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const float rs = 32 * i + lr < rw ? g.rs[mw + 32 * i + lr] : 0.0f;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        uint2 v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t e[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) e[u] = float_to_bf16(acc[i][j][4 * q + u] * rs);
          v[q] = make_uint2(e[0] | (e[1] << 16), e[2] | (e[3] << 16));
        }
        put(i, j, v);
      }
    }
    flush(g.dX);
  }
}

// Tile height (64, 128 or 256 rows) and splits of the contraction, by the time a
// CU with the most work takes. n workgroups are k = ceil(n / 256) a CU, a share
// `load` of what k on every CU would be; `live` is the share of the tiles' rows
// that exist. A K step costs a workgroup, in us (from sweeps of heights and splits
// at 100 to 2048 rows; more with more CUs busy, as the clock falls):
//             gradients, adapters               dual
//   256 rows  0.39 live + 0.6 load, at least     0.75 + 0.25 load
//             0.66
//   128 rows  0.54, or two and more a CU        0.74, 0.45 + 0.2 live load
//             0.35 + 0.22 live load each
//    64 rows  0.46, 0.38                        0.60, 0.55
// A workgroup costs its prologue and results (3, 2 or 1.5 us) besides, splits
// the partial sums, written and read at 4.5 TB/s, and a kernel that adds them.
// Measured (us): gradient of 150 rows of 11008 x 4096: 256 rows in 2 splits 38.4, 128
// rows 42.9; of 200 rows of 4096 x 4096: 128 rows in 4 splits 24.6, 256 in 8 28.2;
// dual, 150 rows of 11008 x 4096: 256 rows in 4 splits 61.7, 128 in 2 77.4; 777 of
// 5120 x 1536: 256 in 2 splits 56.7, 128 in 3 55.8; 2048 of 4096 x 11008: 801, 543, 497
// with 64, 128, 256 rows. (The model's dual steps are from before the roundings had
// products of their own; over 60 shapes of 70 to 2048 rows with them the plan takes the
// fastest of 30 heights and splits or one within 7 %, at 300 rows within 11 %.)
void plan_tiles(FfnPlan& p, int M, int tiles_n, int nk, size_t sum_cols, bool dual) {
  const int heights[3] = {64, 128, 256};
  const double start[3] = {1.5, 2.0, 3.0};
  double best = 1e30;
  p.tiles_n = tiles_n;
  p.nk = nk;
  for (int h = 0; h < 3; ++h)
    for (int s = 1; s <= 16 && (s == 1 || nk / s >= 2); ++s) {
      const int kper = (nk + s - 1) / s;
      if ((nk + kper - 1) / kper != s) continue;
      const int tiles_m = (M + heights[h] - 1) / heights[h];
      const double n = (double)tiles_m * tiles_n * s;
      const double k = (double)(((long long)n + 255) / 256);
      const double load = n / (256.0 * k);
      const double live = (double)M / ((double)tiles_m * heights[h]);
      double step;
      if (h == 2)
        step = dual ? 0.75 + 0.25 * load : std::max(0.66, 0.39 * live + 0.6 * load);
      else if (h == 1)
        step = k == 1 ? (dual ? 0.74 : 0.54)
                      : (dual ? 0.45 + 0.2 * live * load : 0.35 + 0.22 * live * load);
      else
        step = k == 1 ? (dual ? 0.60 : 0.46) : (dual ? 0.55 : 0.38);
      double cost = k * (kper * step + start[h]);
      if (s > 1) cost += 4.0 + s * (double)M * (double)sum_cols * 8.0 / 4.5e6;
      if (cost < best) {
        best = cost;
        p.BM = heights[h];
        p.tiles_m = tiles_m;
        p.kper = kper;
        p.S = s;
      }
    }
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

template <Side SIDE>
hipError_t launch_tiles(TileArgs& g, const FfnPlan& p, hipStream_t st) {
  g.tiles_n = p.tiles_n;
  g.S = p.S;
  g.kper = p.kper;
  g.nk = p.nk;
  const long long grid = (long long)p.tiles_m * p.tiles_n * p.S;
  if (grid > 0x3fffffLL) return hipErrorInvalidValue;  // below 2^32 lanes
  if (p.BM == 64)
    hipLaunchKernelGGL((ffn_gemm_kernel<64, SIDE>), dim3((unsigned)grid), dim3(kTileThreads<64>), 0, st,
                       g);
  else if (p.BM == 128)
    hipLaunchKernelGGL((ffn_gemm_kernel<128, SIDE>), dim3((unsigned)grid), dim3(kTileThreads<128>), 0, st,
                       g);
  else
    hipLaunchKernelGGL((ffn_gemm_kernel<256, SIDE>), dim3((unsigned)grid), dim3(kTileThreads<256>), 0,
                       st, g);
  return hipGetLastError();
}

}  // namespace

// Up to so many rows go through the strips; of those, most use different
// adapters (requests that decode), and the narrow product is formed row by row.
constexpr int kFewRows = 64;

FfnPlan plan_glu_gemm(int M, int N, int K) {
  FfnPlan p{};
  if (M <= kFewRows) {
    p.strip = true;
    p.sp = plan_strip(M, N, K, 2, false);
    p.S = p.sp.S;
    p.ws_bytes = p.sp.part_bytes;
    return p;
  }
  plan_tiles(p, M, (N + 63) / 64, K / BK, (size_t)2 * N, true);
  p.ws_bytes = p.S > 1 ? (size_t)2 * p.S * M * N * sizeof(float) : 0;
  return p;
}

hipError_t launch_glu_gemm(const uint16_t* X, const uint8_t* Wg, const uint8_t* Wu, uint16_t* H,
                           uint16_t* G, uint16_t* U, int M, int N, int K, int act, void* ws,
                           const FfnPlan& p, hipStream_t st) {
  if (p.strip) {
    float* part = static_cast<float*>(ws);
    const hipError_t err = launch_strip(X, Wg, Wu, part, M, N, K, false, p.sp, st);
    if (err != hipSuccess) return err;
    return launch_glu_finish_f16(part, H, G, U, (size_t)M * N, p.S, act, st);
  }
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

FfnPlan plan_gemm_lora(int M, int N, int K, int R) {
  FfnPlan p{};
  p.strip = M <= kFewRows;
  if (p.strip) {
    p.sp = plan_strip(M, N, K, 1, false);
    p.S = p.sp.S;
  } else {
    plan_tiles(p, M, (N + BN - 1) / BN, K / BK, (size_t)N, false);
  }
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at = align256(at + bytes);
    return o;
  };
  if (!p.strip) p.off_tp = take((size_t)shrink_shares(M, K) * M * R * sizeof(float));
  if (p.strip || p.S > 1) {
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
  const bool sums = p.strip || p.S > 1;  // partial sums, finished by lora_finish
  float* part = reinterpret_cast<float*>(w + p.off_part);
  float* t = sums ? reinterpret_cast<float*>(w + p.off_t) : nullptr;
  uint16_t* t16 = sums ? nullptr : reinterpret_cast<uint16_t*>(w + p.off_t16);
  float* ts = sums ? nullptr : reinterpret_cast<float*>(w + p.off_ts);
  if (p.strip) {
    const hipError_t err = launch_strip(X, B, nullptr, part, M, N, K, false, p.sp, st, &ad, t);
    if (err != hipSuccess) return err;
    return launch_lora_finish_f16(part, t, ad, Y, M, N, p.S, st);
  }
  float* tp = reinterpret_cast<float*>(w + p.off_tp);
  hipError_t err = launch_lora_shrink(X, ad, tp, t, t16, ts, M, K, st);
  if (err != hipSuccess) return err;
  TileArgs g{};
  g.X = X;
  g.W0 = B;
  g.M = M;
  g.ncols = N;
  g.lda = K;
  g.NB = N / kBlockWeights;
  g.wrows = K;
  g.part = part;
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
  plan_tiles(p, M, (K + BN - 1) / BN, mats * (N / BK), (size_t)K, false);
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
