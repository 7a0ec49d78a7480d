// Backward pass of the weightless linear from an 8-bit activation checkpoint.
//
// Forward: y = s (.) (x W0^T) + (x V) U^T, the rows of a stacked call's
// children concatenated.  With X the values of the checkpoint (code * 2^e,
// bf16 exactly) and dy the output's gradient:
//
//   z = X V,  g = dy U                      (thin products)
//   dx  = (dy (.) s) W0 + g V^T
//   G   = dy^T X                            (fp32, never stored)
//   dW0 = diag(s) G        ds_n = sum_k G[n][k] W0[n][k]
//   dU  = dy^T z           dV = X^T g
//
// ds needs y's shared part only through G: sum_t dy[t][n] (x W0^T)[t][n] =
// sum_k G[n][k] W0[n][k], so one product gives both dW0 and ds and the
// forward product is not recomputed.
//
// Every product is C[b][a] = sum_c A(a, c) B(b, c) with the output's
// contiguous dimension on the A side (the MFMA's rows: a lane holds four
// consecutive a of one b).  An operand is stored either with c contiguous
// ("k-rows": row a holds its c's) or with a contiguous ("k-columns": row c
// holds all a's, as W0, V^T and U are for dx and g, and dy and X for G).
// Both come from HBM straight into LDS as they lie; a k-column operand is
// transposed on its way to the registers by ds_read_b64_tr_b16, so no
// transposed copy of a weight is ever written (of dy and X only where few
// tokens make it small: few_kernel).
//
// What is rounded on the way, as the matrix cores take bf16 operands: dy (.) s
// once to bf16, and z and g to a pair of bf16 (the value and what its rounding
// left, 16 significant bits, as decode keeps z), which enter their products as
// two runs of the contraction: with one bf16 the errors of dU and dV against
// 64 bits were 1.5 times those of rounding the results alone.  G is exact
// products of bf16 values summed in fp32, and dW0 and ds stay fp32.
#include <algorithm>
#include <type_traits>

#include "coded.h"
#include "common.h"
#include "lds_dma.h"
#include "training.h"

namespace wl {

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;

constexpr int kStep = 64;  // contraction values a product is planned and split in
constexpr int kCUs = 256;
constexpr int kMaxSeg = 5;  // dx: dy's slots (q, k and a tied v), then the pair of g
constexpr int kMaxProb = 1 + 3 * kMaxChildren;  // dx; G, dU and dV of every child
constexpr int kGroupN = 8;  // output tiles along b that run together

// A run of the contraction: A and B hold `len` values of it.
struct Seg {
  const uint16_t *A, *B;
  int64_t lda, ldb;
  int32_t len;
};

// How the operands lie: A and B k-rows; A k-columns, B k-rows; both k-columns.
enum Kind : int32_t { kRowsRows = 0, kColsRows = 1, kColsCols = 2 };
// What becomes of C: bf16 rows, a pair of bf16 rows, or (G) dW0 and ds.
enum ProbMode : int32_t { kBf16 = 0, kPair = 1, kWeight = 2 };

// One product C[N][M] of a launch.
struct Prob {
  Seg seg[kMaxSeg];
  int32_t nseg;
  int32_t M, N;       // extent along A (contiguous in C) and along B
  int32_t kind, mode;
  int32_t nM, nN, ksplit, per;  // tiles, slices of the contraction, steps per slice
  uint16_t *out;      // kBf16, kPair: [N][ldo]
  int64_t ldo;
  int32_t lo;         // kPair: columns from a value to what its rounding left
  float *P;           // ksplit > 1: partials [ksplit][N][ldp]
  int32_t ldp;
  // kWeight: G's consumers
  const float *s;     // [N]
  const uint16_t *W0; // [N][M]
  float *dw0;         // [N][M] or null
  int32_t accumulate;
  float *ds;          // [N] (null: not wanted)
  float *dsp;         // ksplit == 1: its partial sums [nM * 2][ldds], a row per half of a column tile
  int32_t ldds;
};

struct BwdArgs {
  int32_t nprob, total;
  int32_t unit0[kMaxProb];  // first workgroup of each product (behind the last: kNoUnit)
  Prob p[kMaxProb];
};
constexpr int32_t kNoUnit = 0x7fffffff;

// A uniform value held in a scalar register: without it the compiler loads a
// kernel argument again at every use, and a scalar load in the loop makes the
// next use wait for every LDS read in flight (they share a counter).
__device__ __forceinline__ int keep(int v) { return __builtin_amdgcn_readfirstlane(v); }

// One operand of a staged product: W rows of the tile by BK (32 or 64) of the
// contraction per stage, in 1 KB load instructions.
//
// k-rows (TR false, BK = 64): LDS row r is the 64 values of tile row r, its
// 16-byte chunk c in slot c ^ (r % 8): a fragment read (8 lanes per phase: 8
// rows, one chunk) then touches every bank once.
//
// k-columns (TR): LDS row k is W elements of contraction index k, its chunk c
// in slot c ^ swz(k).  A transposing read takes 32-byte pieces of rows 8 g +
// 0..3 (lane group g); two lane groups at once touch 8 rows, which the swizzle
// puts in 8 different 32-byte places of the 256-byte bank period (every row
// starts at bank 0): swz = 2 (k & 3) + 8 (k >> 3 & 1).
//
// A lane's place in a load is a per-lane part (kept in two registers) and a
// part of the instruction's number, so the addresses of the loads cost no
// registers of their own.
template <int W, bool TR, int BK>
struct Operand {
  static constexpr int READS = TR ? 2 : 1;          // LDS reads of a fragment
  static constexpr int CPR = TR ? W / 8 : BK / 8;       // 16-byte chunks of an LDS row
  static constexpr int RPQ = 64 / CPR;              // LDS rows of a load instruction
  static_assert(TR ? W == 128 || W == 256 : BK == 64, "operand shape");

  int lrow, chunk;   // this lane's row of a load and its chunk, without the instruction's swizzle
  uint32_t lo;       // byte offset of lrow's start
  int rd;            // fragment reads: byte offset of the lane's first row
  int sq;            // bytes from a load instruction's rows to the next's (uniform)

  // mw: the wave's first row of the tile
  __device__ __forceinline__ Operand(int lane, int64_t ld, int mw) {
    const int r16 = lane & 15, g = lane >> 4;
    lrow = lane / CPR;
    sq = keep(static_cast<int>(RPQ * ld * 2));
    lo = static_cast<uint32_t>(lrow * ld * 2);
    const int slot = lane % CPR;
    if constexpr (TR) {
      chunk = slot ^ (2 * (lrow & 3));
      const int k = 8 * g + (r16 >> 2);
      const int sw = 2 * (k & 3) + 8 * ((k >> 3) & 1);
      rd = k * (2 * W) + (((mw / 8 + ((r16 >> 1) & 1)) ^ sw) * 16) + (r16 & 1) * 8;
    } else {
      chunk = slot ^ (lrow & 7);
      rd = (mw + r16) * (2 * BK) + (g ^ (r16 & 7)) * 16;
    }
  }
  // Swizzle part of load instruction q (the bits of its first row).
  static __device__ __forceinline__ int sw_of(int q) {
    if constexpr (!TR) return 0;
    return W == 256 ? 4 * (q & 1) + 8 * ((q >> 2) & 1) : 8 * ((q >> 1) & 1);
  }
  // Load instruction q of a stage at `base`; lim rows (k-rows) or columns
  // (k-columns) of the tile exist, `left` values of the contraction.
  __device__ __forceinline__ void load(const uint16_t *base, int q, int lim, int left, lds_u8 *dst) const {
    const int c = chunk ^ sw_of(q), row = q * RPQ + lrow;
    const bool in = TR ? c * 8 < lim && row < left : row < lim && c * 8 < left;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(tile_rsrc(base), (lds_void *)(dst + q * 1024), 16,
                                             in ? lo + c * 16 : kBufNoRow, q * sq, 0, 0);
  }
  static __device__ __forceinline__ const uint16_t *base(const uint16_t *p, int64_t ld, int m0, int k) {
    return TR ? p + k * ld + m0 : p + m0 * ld + k;
  }
  static __device__ __forceinline__ int64_t advance(int64_t ld) { return TR ? BK * ld : BK; }

  // Fragment i (rows 16 i .. of the wave's), contraction 32 h + 8 g .. + 7 in
  // lane group g.  Stages start at multiples of 1 KB, so an exclusive or moves
  // between the chunks of a row.
  __device__ __forceinline__ u32x4 frag(const lds_u8 *lds, int stage, int i, int h) const {
    if constexpr (TR) {
      const lds_u8 *p = lds + ((stage + rd) ^ (32 * i)) + 32 * h * 2 * W;
      const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
      const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 4 * 2 * W));
      const u32x2 x = __builtin_bit_cast(u32x2, a), y = __builtin_bit_cast(u32x2, b);
      return u32x4{x[0], x[1], y[0], y[1]};
    } else {
      return *(const lds_u32x4 *)(lds + ((stage + rd) ^ (64 * h)) + i * 16 * 2 * BK);
    }
  }
};

// NST stages of BK contraction values of a BM x BN tile, on WM x WN waves.
template <int BM_, int BN_, int WM_, int WN_, int BK_, int NST_>
struct BTile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, BK = BK_, NST = NST_;
  static constexpr int NW = WM * WN;
  static constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
  static constexpr int LA = BM * BK / 512 / NW, LB = BN * BK / 512 / NW;  // load instructions of a wave per stage
  static constexpr int LPW = LA + LB;
  static constexpr int BOFF = BM * BK * 2, STAGE = BOFF + BN * BK * 2;    // B behind A in a stage
  static constexpr int PITCH = 2 * BM + 16;      // staged bf16 output: bytes per b
  static constexpr size_t RING = static_cast<size_t>(NST) * STAGE, OUT = static_cast<size_t>(BN) * PITCH;
  static constexpr size_t LDS = RING > OUT ? RING : OUT;
  static_assert(BM * BK / 512 % NW == 0 && BN * BK / 512 % NW == 0 && TM % 16 == 0 && TN % 16 == 0 && LDS <= 160 * 1024, "tile shape");
};

// G's consumers, from the accumulators as they lie (a lane holds k = 16 i +
// 4 g .. + 3 of rows n = 16 j + r16): W0 and dW0 move as 8- and 16-byte pieces
// whose neighbours (i) complete each cache line, all of W0's loads are in
// flight before the first is used, and ds needs two lane exchanges per j.
// (Rows staged through LDS for whole-row accesses took 25 us per 256 x 256
// tile: a load latency and five exchanges for every two rows.)
template <typename TL>
__device__ __forceinline__ void load_block(u32x2 (&w)[TL::FN][TL::FM], const Prob &p, int m0, int n0) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave / TL::WN, wn = wave % TL::WN, r16 = lane & 15, g = lane >> 4;
  const int k0 = m0 + wm * TL::TM + g * 4;  // M % 8 == 0: whole groups of 4
#pragma unroll
  for (int j = 0; j < TL::FN; ++j) {
    const int n = n0 + wn * TL::TN + j * 16 + r16;
    const uint16_t *src = p.W0 + static_cast<int64_t>(n < p.N ? n : 0) * p.M + k0;
#pragma unroll
    for (int i = 0; i < TL::FM; ++i) {
      w[j][i] = u32x2{0u, 0u};
      if (n < p.N && k0 + 16 * i < p.M) w[j][i] = *reinterpret_cast<const u32x2 *>(src + 16 * i);
    }
  }
}

template <typename TL>
__device__ __forceinline__ void store_weight_grad(const f32x4 (&acc)[TL::FM][TL::FN], const u32x2 (&w)[TL::FN][TL::FM], const Prob &p, int f, int m0,
                                                  int n0) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave / TL::WN, wn = wave % TL::WN, r16 = lane & 15, g = lane >> 4;
  const int k0 = m0 + wm * TL::TM + g * 4;  // M % 8 == 0: whole groups of 4
  if (p.dw0) {
#pragma unroll
    for (int j = 0; j < TL::FN; ++j) {
      const int n = n0 + wn * TL::TN + j * 16 + r16;
      if (n >= p.N) continue;
      float *dst = p.dw0 + static_cast<int64_t>(n) * p.M + k0;
      const float sc = p.s[n];
#pragma unroll
      for (int i = 0; i < TL::FM; ++i) {
        if (k0 + 16 * i >= p.M) continue;
        f32x4 o = acc[i][j] * sc;
        if (p.accumulate) o += *reinterpret_cast<const f32x4 *>(dst + 16 * i);
        *reinterpret_cast<f32x4 *>(dst + 16 * i) = o;
      }
    }
  }
  if (p.ds) {
#pragma unroll
    for (int j = 0; j < TL::FN; ++j) {
      const int n = n0 + wn * TL::TN + j * 16 + r16;
      float t = 0.f;
#pragma unroll
      for (int i = 0; i < TL::FM; ++i) {
        const f32x4 v = acc[i][j];  // columns past M hold no G (their operand columns are zeros)
        t += v[0] * __uint_as_float(w[j][i][0] << 16) + v[1] * __uint_as_float(w[j][i][0] & 0xffff0000u) +
             v[2] * __uint_as_float(w[j][i][1] << 16) + v[3] * __uint_as_float(w[j][i][1] & 0xffff0000u);
      }
      t += __shfl_xor(t, 16, 64);
      t += __shfl_xor(t, 32, 64);
      if (g == 0 && n < p.N) p.dsp[static_cast<int64_t>(f * TL::WM + wm) * p.ldds + n] = t;
    }
  }
}

// A bf16 tile in LDS, b-major, then whole 16-byte chunks of output rows, `at`
// columns on.
template <typename TL>
__device__ __forceinline__ void store_rows(const f32x4 (&acc)[TL::FM][TL::FN], const Prob &p, int m0, int n0, int at,
                                           uint8_t *lds) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave / TL::WN, wn = wave % TL::WN, r16 = lane & 15, g = lane >> 4;
#pragma unroll
  for (int j = 0; j < TL::FN; ++j)
#pragma unroll
    for (int i = 0; i < TL::FM; ++i) {
      const int tl = wn * TL::TN + j * 16 + r16, fl = wm * TL::TM + i * 16 + g * 4;
      *reinterpret_cast<uint2 *>(lds + tl * TL::PITCH + fl * 2) =
          make_uint2(pack_bf16(acc[i][j][0], acc[i][j][1]),
                     pack_bf16(acc[i][j][2], acc[i][j][3]));
    }
  __syncthreads();
  constexpr int CPR = TL::BM / 8;
  for (int c = threadIdx.x; c < TL::BN * CPR; c += TL::NW * 64) {
    const int tl = c / CPR, fl = (c % CPR) * 8;
    const int n = n0 + tl, m = m0 + fl;
    if (n >= p.N || m >= p.M) continue;
    const uint4 val = *reinterpret_cast<const uint4 *>(lds + tl * TL::PITCH + fl * 2);
    uint16_t *o = p.out + static_cast<int64_t>(n) * p.ldo + m + at;
    if (m + 8 <= p.M && (reinterpret_cast<uintptr_t>(o) & 15) == 0) {
      *reinterpret_cast<uint4 *>(o) = val;
    } else {
      const uint32_t e[4] = {val.x, val.y, val.z, val.w};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (m + i < p.M) o[i] = static_cast<uint16_t>(e[i / 2] >> (16 * (i & 1)));
    }
  }
}

// Loads of a stage into `w`: all of it, or all but the last instruction (the
// first of its two steps when a stage is two halves deep), or that last one.
enum Part : int { kAll = 0, kFirst = 1, kLast = 2 };

template <typename TL, Part PART, typename OA, typename OB>
__device__ __forceinline__ void load_stage(const OA &oa, const OB &ob, const uint16_t *pa, const uint16_t *pb,
                                           int lima, int limb, int left, int wave,
                                           lds_u8 *w) {
  if constexpr (PART != kLast) {
#pragma unroll
    for (int q = 0; q < TL::LA; ++q) oa.load(pa, wave * TL::LA + q, lima, left, w);
  }
#pragma unroll
  for (int q = 0; q < TL::LB; ++q)
    if (PART == kAll || (PART == kLast) == (q == TL::LB - 1)) ob.load(pb, wave * TL::LB + q, limb, left, w + TL::BOFF);
}

// One pipeline step's memory work: loads of a stage into `w`, and the
// fragments of half h of the stage at r + stage.  They are different stages,
// and saying so (restrict, on accesses of one call) keeps the compiler from
// draining the loads in flight before the transposing reads, whose addresses
// it does not follow (it did: 1.8x the time of a 256 x 256 tile's step).
// What orders a stage's loads before its own reads is the counted wait and
// barrier between them.
template <typename TL, Part PART, typename OA, typename OB>
__device__ __forceinline__ void move_stage(const OA &oa, const OB &ob, const uint16_t *pa, const uint16_t *pb,
                                           int lima, int limb, int left, int wave,
                                           lds_u8 *__restrict__ w, const lds_u8 *__restrict__ r, int stage, int h,
                                           u32x4 (&fa)[TL::FM], u32x4 (&fb)[TL::FN]) {
  load_stage<TL, PART>(oa, ob, pa, pb, lima, limb, left, wave, w);
#pragma unroll
  for (int j = 0; j < TL::FN; ++j) fb[j] = ob.frag(r, stage + TL::BOFF, j, h);
#pragma unroll
  for (int i = 0; i < TL::FM; ++i) fa[i] = oa.frag(r, stage, i, h);
}

// Unit v of product p: a tile of C over one slice of the contraction.
template <typename TL, bool ATR, bool BTR>
__device__ __forceinline__ void product_unit(const Prob &p, int v, uint8_t *lds) {
  using OA = Operand<TL::BM, ATR, TL::BK>;
  using OB = Operand<TL::BN, BTR, TL::BK>;
  lds_u8 *const ring = (lds_u8 *)lds;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / TL::WN, wn = wave % TL::WN;
  const int r16 = lane & 15, g = lane >> 4;
  // kGroupN tiles along b share their A panels, then the next panel, then the
  // next group
  const int sl = v / (p.nM * p.nN), w = v % (p.nM * p.nN);
  const int grp = w / (p.nM * kGroupN), gn = min(kGroupN, p.nN - grp * kGroupN);
  const int wg = w - grp * p.nM * kGroupN;
  const int f = wg / gn, t = grp * kGroupN + wg % gn;
  const int m0 = f * TL::BM, n0 = t * TL::BN;
  int s_lo = sl * p.per, s_hi = s_lo + p.per;  // steps of this slice, counted through the segments

  f32x4 acc[TL::FM][TL::FN];
#pragma unroll
  for (int i = 0; i < TL::FM; ++i)
#pragma unroll
    for (int j = 0; j < TL::FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  u32x2 w0[TL::FN][TL::FM];
  if constexpr (ATR && BTR && TL::BM == 128) {
    if (p.mode == kWeight && p.ksplit == 1 && p.ds) load_block<TL>(w0, p, m0, n0);
  }
  for (int si = 0; si < p.nseg; ++si) {
    const Seg &sg = p.seg[si];
    const int steps = (sg.len + kStep - 1) / kStep;
    const int b0 = max(0, s_lo), ns = min(steps, s_hi) - b0;
    s_lo -= steps;
    s_hi -= steps;
    if (ns <= 0) continue;
    const OA oa(lane, sg.lda, wm * TL::TM);
    const OB ob(lane, sg.ldb, wn * TL::TN);
    const uint16_t *pa = OA::base(sg.A, sg.lda, m0, b0 * kStep), *pb = OB::base(sg.B, sg.ldb, n0, b0 * kStep);
    const int adv_a = keep(static_cast<int>(OA::advance(sg.lda))), adv_b = keep(static_cast<int>(OB::advance(sg.ldb)));
    int left = min(sg.len, (b0 + ns) * kStep) - b0 * kStep;  // values from the next stage to load on
    auto advance = [&]() {
      pa += adv_a;
      pb += adv_b;
      left -= TL::BK;
    };
    auto multiply = [&](const u32x4(&fa)[TL::FM], const u32x4(&fb)[TL::FN]) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < TL::FM; ++i)
#pragma unroll
        for (int j = 0; j < TL::FN; ++j) acc[i][j] = mfma16x16x32(fa[i], fb[j], acc[i][j]);
      interleave_mfma<TL::FM * TL::FN, OA::READS * TL::FM + OB::READS * TL::FN, TL::LPW>();
    };
    // Software pipeline over 32-deep halves: while one is multiplied from
    // registers, the next is read from LDS, and the stages after that are in
    // flight.  A step into a new stage opens with the barrier: there every
    // wave has read all of the stage before, so its buffer takes the loads of
    // the stage NST ahead, and the new stage has landed.  Loads past the last
    // stage read no rows (zeros), so that the loop needs no branches and
    // counts the same loads in flight at every step.
    u32x4 a0[TL::FM], b0f[TL::FN], a1[TL::FM], b1f[TL::FN];
    constexpr bool kHalves = TL::BK == 64;
    const int lima = keep(p.M - m0), limb = keep(p.N - n0);
#pragma unroll
    for (int st = 0; st < TL::NST; ++st) {
      if (kHalves && st == TL::NST - 1) {
        load_stage<TL, kFirst>(oa, ob, pa, pb, lima, limb, left, wave, ring + st * TL::STAGE);
      } else {
        load_stage<TL, kAll>(oa, ob, pa, pb, lima, limb, left, wave, ring + st * TL::STAGE);
        advance();
      }
    }
    wait_and_sync<(TL::NST - 1) * TL::LPW - (kHalves ? 1 : 0)>();
    int cur = 0, old = (TL::NST - 1) * TL::STAGE;  // the stage read, the stage loaded last
#pragma unroll
    for (int j = 0; j < TL::FN; ++j) b0f[j] = ob.frag(ring, TL::BOFF, j, 0);
#pragma unroll
    for (int i = 0; i < TL::FM; ++i) a0[i] = oa.frag(ring, 0, i, 0);
    auto into_stage = [&](u32x4(&fa)[TL::FM], u32x4(&fb)[TL::FN]) __attribute__((always_inline)) {
      wait_and_sync<(TL::NST - 2) * TL::LPW>();
      old = cur;
      cur = cur + TL::STAGE == static_cast<int>(TL::RING) ? 0 : cur + TL::STAGE;
      move_stage<TL, kHalves ? kFirst : kAll>(oa, ob, pa, pb, lima, limb, left, wave, ring + old, ring,
                                              cur, 0, fa, fb);
      if (!kHalves) advance();
    };
    for (int kt = 0; kt < ns; ++kt) {
      if constexpr (kHalves) {
        move_stage<TL, kLast>(oa, ob, pa, pb, lima, limb, left, wave, ring + old, ring, cur, 1, a1, b1f);
        advance();
      } else {
        into_stage(a1, b1f);
      }
      multiply(a0, b0f);
      into_stage(a0, b0f);
      multiply(a1, b1f);
    }
    wait_and_sync<0>();  // the ring is idle
  }

  if (p.ksplit > 1) {
    float *P = p.P + static_cast<int64_t>(sl) * p.N * p.ldp;
#pragma unroll
    for (int j = 0; j < TL::FN; ++j) {
      const int n = n0 + wn * TL::TN + j * 16 + r16;
      if (n >= p.N) continue;
#pragma unroll
      for (int i = 0; i < TL::FM; ++i) {
        const int m = m0 + wm * TL::TM + i * 16 + g * 4;
        if (m < p.ldp) *reinterpret_cast<f32x4 *>(P + static_cast<int64_t>(n) * p.ldp + m) = acc[i][j];
      }
    }
    return;
  }
  if (p.mode == kWeight) {
    if constexpr (ATR && BTR) {
      if constexpr (TL::BM != 128) {
        if (p.ds) load_block<TL>(w0, p, m0, n0);
      }
      store_weight_grad<TL>(acc, w0, p, f, m0, n0);
    }
    return;
  }
  store_rows<TL>(acc, p, m0, n0, 0, lds);
  if constexpr (TL::BM == 128) {  // pairs are planned on these tiles only
    if (p.mode != kPair) return;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < TL::FN; ++j)
#pragma unroll
      for (int i = 0; i < TL::FM; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] -= bf16_to_f32(f32_to_bf16(acc[i][j][e]));
    store_rows<TL>(acc, p, m0, n0, p.lo, lds);
  }
}

// Workgroup -> product and its unit.  The units of each product are numbered
// XCD-major, so that the tiles an XCD runs at a time share panels in its L2.
__device__ __forceinline__ const Prob &find_unit(const BwdArgs &a, int &v) {
  int pi = 0, first = 0;
#pragma unroll
  for (int i = 1; i < kMaxProb; ++i)  // (one run of arguments: no chain of loads)
    if (static_cast<int>(blockIdx.x) >= a.unit0[i]) {
      pi = i;
      first = a.unit0[i];
    }
  const Prob &p = a.p[pi];
  v = xcd_unit(blockIdx.x - first, p.nM * p.nN * p.ksplit);
  return p;
}

template <typename TL, bool ATR, bool BTR>
__global__ __launch_bounds__(TL::NW * 64) __attribute__((amdgpu_waves_per_eu(1, 2))) void product_kernel(BwdArgs args) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  int v;
  const Prob &p = find_unit(args, v);
  product_unit<TL, ATR, BTR>(p, v, lds);
}

// Products of any kind in one launch.
template <typename TL>
__global__ __launch_bounds__(TL::NW * 64) __attribute__((amdgpu_waves_per_eu(1, 4))) void products_kernel(BwdArgs args) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  int v;
  const Prob &p = find_unit(args, v);
  if (p.kind == kColsCols)
    product_unit<TL, true, true>(p, v, lds);
  else if (p.kind == kColsRows)
    product_unit<TL, true, false>(p, v, lds);
  else
    product_unit<TL, false, false>(p, v, lds);
}

// Few tokens (T <= 128): dx, dW0 and ds in one pass over W0.  A workgroup
// owns 128 columns k and a slice of the rows n of W0; a stage is 64 rows.  From
// it come dx's terms, with the 64 columns of dy (.) s that belong to the rows,
// and the stage's G, whose contraction is the tokens alone: dy and X are at hand
// transposed, in panels of 64 tokens [column][64], so G's operands need no LDS
// transpose and X's stay in registers.  For dx a wave takes 16 k and all n, for
// G 64 k and 16 n.  dx's other terms (g V^T) are further stages without G.
// Bound by W0 once through and dW0's way out (43008 x 5376 at T = 16: 273 us,
// 5.1 TB/s; the counted wait on a stage also waits out dW0 stores of the steps
// before).  Without dW0 bound by a step's own chain -- barrier, LDS reads,
// MFMAs, ds's lane exchanges in turn, nothing read ahead -- of which a
// workgroup runs 115, 1.15 us each (133 us, 3.5 TB/s): matrix cores busy 0.20
// and LDS 0.24 of the cycles, waves waiting 0.47.  A step does 64 tokens' work
// for any T <= 64.  Past 64 tokens a stage holds two panels and the ring three
// stages (the call at T = 128: 596 -> 430 us, without dW0 391 -> 292; the pass
// then 0.25, 0.23 and 0.47); three panels would leave no ring.
constexpr int kPanel = 64, kFewPanels = 2, kFewWaves = 8;

// H panels of tokens.
template <int H_>
struct FewTile {
  static constexpr int H = H_, T = H * kPanel, NST = H == 1 ? 4 : 3;
  static constexpr int Y = 64 * 128 * 2, D = Y + T * 128, S = D + 64 * 2 * T;  // in a stage: dy (.) s, dy^T, s
  static constexpr int STAGE = S + kFewWaves * 256, RING = NST * STAGE;
  static constexpr int LPW = 2 + 2 * H + 1;  // load instructions of a wave per stage
  static_assert(RING <= 160 * 1024, "ring");
};

struct FewArgs {
  Prob p;  // dx: M = K, N = T; its segments over dy's slots come first
  int32_t nslot;
  int32_t row[kMaxChildren];          // slot -> first row of W0, s, dW0 and ds
  const uint16_t *dyt[kMaxChildren];  // slot -> dy^T [panel][columns][64]
  const uint16_t *xt;                 // X^T [panel][K][64]
  int64_t dpanel;                     // elements from a panel of dy^T to the next
};

template <typename TL>
struct FewOperands {
  Operand<128, true, 64> a;       // W0 (or V^T): 128 columns
  Operand<TL::T, false, 64> b;    // dy (.) s (or g): the tokens
  Operand<64, false, 64> d;       // dy^T: the stage's rows n
};

struct FewSource {
  const uint16_t *a, *b, *d;
  const float *s;
  int64_t dpanel;
  int lima, limb, left, leftd;  // columns, tokens; rows n left, of them with a G
};

template <typename TL>
struct FewFrags {
  u32x4 a[2], b[TL::T / 16][2], d[TL::H][2];
  u32x2 w[4];
  float s;
};

// A stage's loads into `w` and another's reads from `r` (restrict: move_stage).
template <typename TL>
__device__ __forceinline__ void few_load(const FewOperands<TL> &o, const FewSource &f, int lane, int wave, lds_u8 *w) {
  o.a.load(f.a, 2 * wave, f.lima, f.left, w);
  o.a.load(f.a, 2 * wave + 1, f.lima, f.left, w);
#pragma unroll
  for (int h = 0; h < TL::H; ++h) {
    o.b.load(f.b, TL::H * wave + h, f.limb, f.left, w + TL::Y);
    o.d.load(f.d + h * f.dpanel, wave, f.leftd, kPanel, w + TL::D + h * 64 * 2 * kPanel);
  }
  __builtin_amdgcn_raw_ptr_buffer_load_lds(tile_rsrc(f.s), (lds_void *)(w + TL::S + wave * 256), 4,
                                           lane < f.leftd ? lane * 4 : kBufNoRow, 0, 0, 0);
}

template <typename TL>
__device__ __forceinline__ void few_step(const FewOperands<TL> &o, const FewSource &f, int lane, int wave,
                                         lds_u8 *__restrict__ w, const lds_u8 *__restrict__ r, int stage,
                                         FewFrags<TL> &x) {
  few_load<TL>(o, f, lane, wave, w);
  const int r16 = lane & 15, g = lane >> 4, n = (wave & 3) * 16 + r16;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    x.a[h] = o.a.frag(r, stage, 0, h);
#pragma unroll
    for (int j = 0; j < TL::T / 16; ++j) x.b[j][h] = o.b.frag(r, stage + TL::Y, j, h);
#pragma unroll
    for (int q = 0; q < TL::H; ++q) x.d[q][h] = o.d.frag(r, stage + TL::D + q * 64 * 2 * kPanel, wave & 3, h);
  }
  // W0[n][64 (wave / 4) + 16 i + 4 g ..]: chunk c of LDS row n lies in slot c ^ swz(n)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = (wave >> 2) * 8 + 2 * i + (g >> 1), swz = 2 * (n & 3) + 8 * ((n >> 3) & 1);
    x.w[i] = *(const __attribute__((address_space(3))) u32x2 *)(r + stage + n * 256 + ((c ^ swz) * 16) + (g & 1) * 8);
  }
  x.s = *(const __attribute__((address_space(3))) float *)(r + stage + TL::S + wave * 256 + n * 4);
}

template <typename TL>
__global__ __launch_bounds__(kFewWaves * 64) __attribute__((amdgpu_waves_per_eu(1, 2))) void few_kernel(FewArgs args) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  lds_u8 *const ring = (lds_u8 *)lds;
  const Prob &p = args.p;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int v = xcd_unit(blockIdx.x, p.nM * p.ksplit);
  const int sl = v / p.nM, f = v % p.nM, m0 = f * 128;
  const bool want_x = p.out != nullptr, want_g = p.ds || p.dw0;
  int s_lo = sl * p.per, s_hi = s_lo + p.per;
  const int kg = m0 + (wave >> 2) * 64;  // G: this wave's columns
  u32x4 xt[4][2 * TL::H];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int h = 0; h < 2 * TL::H; ++h) {
      const int k = kg + 16 * i + r16;
      xt[i][h] = u32x4{0u, 0u, 0u, 0u};
      if (want_g && k < p.M)
        xt[i][h] = ld16(args.xt + (static_cast<int64_t>(h / 2) * p.M + k) * kPanel + 32 * (h % 2) + 8 * g);
    }
  f32x4 acc[TL::T / 16];
#pragma unroll
  for (int j = 0; j < TL::T / 16; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};

  for (int si = 0; si < p.nseg; ++si) {
    const Seg &sg = p.seg[si];
    const int steps = (sg.len + kStep - 1) / kStep;
    const int b0 = max(0, s_lo), ns = min(steps, s_hi) - b0;
    s_lo -= steps;
    s_hi -= steps;
    if (ns <= 0) continue;
    const bool with_g = want_g && si < args.nslot;
    const FewOperands<TL> o{{lane, sg.lda, wave * 16}, {lane, sg.ldb, 0}, {lane, kPanel, 0}};
    const int64_t n0 = static_cast<int64_t>(b0) * kStep;
    const int64_t row = with_g ? args.row[si] + n0 : 0;
    FewSource src;
    src.a = sg.A + n0 * sg.lda + m0;
    src.b = sg.B + n0;
    src.d = with_g ? args.dyt[si] + n0 * kPanel : sg.B;
    src.dpanel = with_g ? args.dpanel : 0;
    src.s = p.s + row;
    src.lima = keep(want_x || (with_g && p.ds) ? p.M - m0 : 0);
    src.limb = keep(want_x ? p.N : 0);
    src.left = min(sg.len, (b0 + ns) * kStep) - b0 * kStep;
    const int adv_a = keep(static_cast<int>(kStep * sg.lda));
    int rows = src.left;  // of the stage computed and after it
    auto advance = [&]() {
      src.a += adv_a;
      src.b += kStep;
      src.d += kStep * kPanel;
      src.s += kStep;
      src.left -= kStep;
      src.leftd = with_g ? src.left : 0;
    };
    src.leftd = with_g ? src.left : 0;
#pragma unroll
    for (int st = 0; st < TL::NST - 1; ++st) {
      few_load<TL>(o, src, lane, wave, ring + st * TL::STAGE);
      advance();
    }
    int cur = 0, nxt = (TL::NST - 1) * TL::STAGE;
    for (int kt = 0; kt < ns; ++kt) {
      // the stage has landed, and every wave is done with the one before
      wait_and_sync<(TL::NST - 2) * TL::LPW>();
      FewFrags<TL> x;
      few_step<TL>(o, src, lane, wave, ring + nxt, ring, cur, x);
      advance();
      if (want_x) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < TL::T / 16; ++j) acc[j] = mfma16x16x32(x.a[h], x.b[j][h], acc[j]);
      }
      if (with_g) {
        const int n = (wave & 3) * 16 + r16;
        const int64_t at = row + static_cast<int64_t>(kt) * kStep + n;
        const bool in = n < rows;
        float t = 0.f;
        f32x4 G[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          G[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int h = 0; h < 2 * TL::H; ++h) G[i] = mfma16x16x32(xt[i][h], x.d[h / 2][h % 2], G[i]);
        }
        if (p.dw0 && in) {
          float *dst = p.dw0 + at * p.M + kg + 4 * g;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (kg + 16 * i + 4 * g >= p.M) continue;
            f32x4 q = G[i] * x.s;
            if (p.accumulate) q += *reinterpret_cast<const f32x4 *>(dst + 16 * i);
            *reinterpret_cast<f32x4 *>(dst + 16 * i) = q;
          }
        }
        if (p.ds) {
#pragma unroll
          for (int i = 0; i < 4; ++i)  // columns past M: X^T is zero
            t += G[i][0] * __uint_as_float(x.w[i][0] << 16) + G[i][1] * __uint_as_float(x.w[i][0] & 0xffff0000u) +
                 G[i][2] * __uint_as_float(x.w[i][1] << 16) + G[i][3] * __uint_as_float(x.w[i][1] & 0xffff0000u);
          t += __shfl_xor(t, 16, 64);
          t += __shfl_xor(t, 32, 64);
          if (g == 0 && in) p.dsp[static_cast<int64_t>(2 * f + (wave >> 2)) * p.ldds + at] = t;
        }
      }
      rows -= kStep;
      nxt = cur;
      cur = cur + TL::STAGE == TL::RING ? 0 : cur + TL::STAGE;
    }
    wait_and_sync<0>();  // the ring is idle
  }
  if (!want_x) return;
  const int k = m0 + wave * 16 + 4 * g;
  if (k >= p.M) return;
#pragma unroll
  for (int j = 0; j < TL::T / 16; ++j) {
    const int t = 16 * j + r16;
    if (t >= p.N) continue;
    if (p.ksplit > 1)
      *reinterpret_cast<f32x4 *>(p.P + (static_cast<int64_t>(sl) * p.N + t) * p.ldp + k) = acc[j];
    else
      *reinterpret_cast<uint2 *>(p.out + t * p.ldo + k) =
          make_uint2(pack_bf16(acc[j][0], acc[j][1]), pack_bf16(acc[j][2], acc[j][3]));
  }
}

// What is left after the products, one launch: for a split product the sum of
// its slices' partials in slice order -- rows of C as bf16 or a pair (a thread
// per 4 elements), or dW0's row and ds[n] (a workgroup per row n of G) -- and
// for an unsplit G ds from its column tiles' partial sums (16 rows n per
// workgroup, 16 lanes per row each summing every 16th part, joined in order).
struct SumArgs {
  int32_t nprob;
  int32_t first[kMaxProb];  // first workgroup of each (behind the last: kNoUnit)
  Prob p[kMaxProb];
};

static_assert(sizeof(BwdArgs) <= 4096 && sizeof(SumArgs) <= 4096, "kernel arguments");

__device__ __forceinline__ f32x4 sum_slices(const Prob &p, int64_t n, int m) {
  f32x4 s{0.f, 0.f, 0.f, 0.f};
  for (int i = 0; i < p.ksplit; ++i)
    s += *reinterpret_cast<const f32x4 *>(p.P + (static_cast<int64_t>(i) * p.N + n) * p.ldp + m);
  return s;
}

__global__ __launch_bounds__(256) void sum_kernel(SumArgs a) {
  int pi = 0;
#pragma unroll
  for (int i = 1; i < kMaxProb; ++i)
    if (static_cast<int>(blockIdx.x) >= a.first[i]) pi = i;
  const Prob &p = a.p[pi];
  const int64_t b = blockIdx.x - a.first[pi];
  const int q = p.ldp / 4;
  if (p.ksplit == 1) {
    const int c = threadIdx.x & 15, l = threadIdx.x >> 4;
    const int64_t n = b * 16 + c;
    float t = 0.f;
    if (n < p.N)
      for (int i = l; i < 2 * p.nM; i += 16) t += p.dsp[static_cast<int64_t>(i) * p.ldds + n];
    __shared__ float part[16][17];
    part[l][c] = t;
    __syncthreads();
    if (threadIdx.x < 16 && n < p.N) {
      t = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) t += part[i][c];
      p.ds[n] = t;
    }
    return;
  }
  if (p.mode != kWeight) {
    const int64_t id = b * 256 + threadIdx.x;
    if (id >= static_cast<int64_t>(p.N) * q) return;
    const int64_t n = id / q;
    const int m = static_cast<int>(id % q) * 4;
    f32x4 s = sum_slices(p, n, m);
    for (int pass = 0; pass < (p.mode == kPair ? 2 : 1); ++pass) {
      uint32_t v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = f32_to_bf16(s[e]);
      uint16_t *o = p.out + n * p.ldo + m + pass * p.lo;
      if (m + 4 <= p.M && (reinterpret_cast<uintptr_t>(o) & 7) == 0) {
        *reinterpret_cast<uint2 *>(o) = make_uint2(v[0] | (v[1] << 16), v[2] | (v[3] << 16));
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (m + e < p.M) o[e] = static_cast<uint16_t>(v[e]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] -= bf16_to_f32(static_cast<uint16_t>(v[e]));
    }
    return;
  }
  const int64_t n = b;
  const float sc = p.s[n];
  float t = 0.f;
  for (int c = threadIdx.x; c < q; c += 256) {
    const f32x4 s = sum_slices(p, n, c * 4);
    if (p.dw0) {
      f32x4 *d = reinterpret_cast<f32x4 *>(p.dw0 + n * p.M + c * 4);
      f32x4 o = s * sc;
      if (p.accumulate) o += *d;
      *d = o;
    }
    if (p.ds) {
      const u32x2 w = *reinterpret_cast<const u32x2 *>(p.W0 + n * p.M + c * 4);
      t += s[0] * __uint_as_float(w[0] << 16) + s[1] * __uint_as_float(w[0] & 0xffff0000u) +
           s[2] * __uint_as_float(w[1] << 16) + s[3] * __uint_as_float(w[1] & 0xffff0000u);
    }
  }
  if (!p.ds) return;
  __shared__ float part[4];
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) t += __shfl_xor(t, d, 64);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = t;
  __syncthreads();
  if (threadIdx.x == 0) p.ds[n] = (part[0] + part[1]) + (part[2] + part[3]);
}

// dy [T][ldy] -> rows of ldd columns in which every child's slot starts at a
// multiple of 8 (zeros behind a slot's last column): the plain copy `dyp`
// and/or dy (.) s rounded to bf16, `dys`; and the checkpoint's values X (bf16
// [T][K]).  One launch: workgroups run along a group of tokens, its first dyb
// take dy, the others X.  Bound by memory: the 31B gate|up call's 390 MB at
// T = 2048 in 61 us (105 with s loaded element by element).
struct PrepArgs {
  const uint16_t *dy;
  int32_t T, ldy, ldd, nslot;
  int32_t start[kMaxChildren + 1];  // slot -> first column in the padded rows (start[nslot] = ldd)
  int32_t from[kMaxChildren];       // slot -> first column in dy
  int32_t n[kMaxChildren];          // slot -> columns
  const float *s[kMaxChildren];
  uint16_t *dyp, *dys;
  int32_t dyb, cols;  // workgroups across dy's columns, and across all columns
  CodedView xc;
  int32_t K;
  uint16_t *X;
  uint16_t *dyt, *xt;  // few tokens: dy^T [panel][ldd][64] and X^T [panel][K][64], zeros past T (else null)
};

// 8 columns of kPrepT tokens as kPrepT tokens of 8 columns
__device__ __forceinline__ void store_transposed(const u32x4 (&v)[4], uint16_t *p) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    uint32_t e[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) e[t] = k & 1 ? v[t][k / 2] >> 16 : v[t][k / 2] & 0xffffu;
    *reinterpret_cast<uint2 *>(p + k * kPanel) = make_uint2(e[0] | (e[1] << 16), e[2] | (e[3] << 16));
  }
}

// A thread takes 8 columns of kPrepT tokens: s is read once for all of them (2
// tokens 66 us, 8 115).
constexpr int kPrepT = 4;

__global__ __launch_bounds__(256) void prepare_kernel(PrepArgs a) {
  const int col = blockIdx.x % a.cols;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x / a.cols) * kPrepT;
  if (col >= a.dyb) {
    const int k = ((col - a.dyb) * 256 + threadIdx.x) * 8;
    if (k >= a.K) return;
    u32x4 v[kPrepT];
#pragma unroll
    for (int i = 0; i < kPrepT; ++i) {
      const int64_t t = t0 + i;
      v[i] = u32x4{0u, 0u, 0u, 0u};
      if (t < a.T) {
        v[i] = expand8(a.xc, t, k);
        *reinterpret_cast<u32x4 *>(a.X + t * a.K + k) = v[i];
      }
    }
    if (a.xt) store_transposed(v, a.xt + (t0 / kPanel * a.K + k) * kPanel + t0 % kPanel);
    return;
  }
  const int c = (col * 256 + threadIdx.x) * 8;
  if (c >= a.ldd) return;
  int i = 0;
  while (i + 1 < a.nslot && c >= a.start[i + 1]) ++i;
  const int j = c - a.start[i], n = a.n[i] - j;  // n: columns of the slot from here on (>= 1)
  float s[8];
  if (a.dys && n >= 8) {  // a slot's s starts at any row: 4-byte aligned
    typedef f32x4 __attribute__((aligned(4))) f32x4_any;
    const f32x4 lo = *reinterpret_cast<const f32x4_any *>(a.s[i] + j), hi = *reinterpret_cast<const f32x4_any *>(a.s[i] + j + 4);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      s[k] = lo[k];
      s[4 + k] = hi[k];
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) s[k] = a.dys && k < n ? a.s[i][j + k] : 0.f;
  }
  const uint16_t *src = a.dy + t0 * a.ldy + a.from[i] + j;
  const int nt = static_cast<int>(min<int64_t>(kPrepT, a.T - t0));  // (past T: none)
  u32x4 v[kPrepT];
#pragma unroll
  for (int t = 0; t < kPrepT; ++t) v[t] = u32x4{0u, 0u, 0u, 0u};
  if (n >= 8 && a.ldy % 8 == 0 && (reinterpret_cast<uintptr_t>(src) & 15) == 0) {
#pragma unroll
    for (int t = 0; t < kPrepT; ++t)
      if (t < nt) v[t] = ld16(src + static_cast<int64_t>(t) * a.ldy);
  } else {
#pragma unroll
    for (int t = 0; t < kPrepT; ++t)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint16_t *q = src + static_cast<int64_t>(t) * a.ldy + 2 * k;
        const uint32_t lo = t < nt && 2 * k < n ? q[0] : 0u, hi = t < nt && 2 * k + 1 < n ? q[1] : 0u;
        v[t][k] = lo | (hi << 16);
      }
  }
  if (a.dyt) store_transposed(v, a.dyt + (t0 / kPanel * a.ldd + c) * kPanel + t0 % kPanel);
#pragma unroll
  for (int t = 0; t < kPrepT; ++t) {
    if (t >= nt) break;
    const int64_t at = (t0 + t) * a.ldd + c;
    if (a.dyp) *reinterpret_cast<u32x4 *>(a.dyp + at) = v[t];
    if (a.dys) {
      u32x4 o;
#pragma unroll
      for (int k = 0; k < 4; ++k)  // columns past the slot: dy and s are 0
        o[k] = pack_bf16(__uint_as_float(v[t][k] << 16) * s[2 * k], __uint_as_float(v[t][k] & 0xffff0000u) * s[2 * k + 1]);
      *reinterpret_cast<u32x4 *>(a.dys + at) = o;
    }
  }
}

__global__ __launch_bounds__(256) void zero_kernel(uint16_t *p, int64_t n) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * 256)
    p[i] = 0;
}

hipError_t launch_zero(void *p, int64_t halves, hipStream_t stream) {
  if (!p || halves <= 0) return hipSuccess;
  const int64_t blocks = std::min<int64_t>((halves + 255) / 256, 4096);
  hipLaunchKernelGGL(zero_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream, static_cast<uint16_t *>(p),
                     halves);
  return hipGetLastError();
}

// ---- host side --------------------------------------------------------------

// 256 x 256 tiles, a launch per kind (A is k-columns).  Stage depth by B: k-column
// rows are long whatever the depth, so four shallow stages keep more loads in
// flight; a k-row operand wants whole 128-byte lines (with 64-byte rows a bare
// load loop ran at 57 KB/us per CU instead of 92).
template <bool BTR>
using Big = std::conditional_t<BTR, BTile<256, 256, 2, 4, 32, 4>, BTile<256, 256, 2, 4, 64, 2>>;
// 128 x 128 tiles, every kind in one launch: with a ring of two stages two
// workgroups share a CU, with four one keeps as many loads in flight.
using Mid2 = BTile<128, 128, 2, 4, 64, 2>;
using Mid4 = BTile<128, 128, 2, 4, 64, 4>;

// Elements of W0 from which few tokens take one pass over it: below, its own
// launch costs more than the second read (43008 x 5376 at T = 16: 536 -> 341 us,
// without dW0 315 -> 195; 5376 x 8192 111 -> 96, 85 -> 66; 8192 x 1152 49 -> 55,
// 40 -> 47).
constexpr int64_t kFewBlock = 16 << 20;

struct BPlan {
  bool big;
  int ksplit, per, nM, nN;
  size_t partial_bytes(int M, int N) const {
    return ksplit > 1 ? (static_cast<size_t>(ksplit) * N * ((M + 3) & ~3) * 4 + 255) & ~size_t{255} : 0;
  }
};

// A product as the planner sees it: extents and contraction steps.
struct Item {
  int M, N, steps;
  bool pair;  // z and g: 128 x 128 tiles only, which store pairs
};

// Microseconds (fitted to the 31B and 1B shapes): a step and the fixed part of
// a 256 x 256 workgroup, of a 128 x 128 workgroup alone on its CU and of one
// of two that share it; bytes per us of the partials' way out and back.
constexpr double kBigStep = 1.7, kBigFix = 10.0;
constexpr double kMidStep = 0.6, kMidPairStep = 1.0, kMidFix = 4.0;
constexpr double kSumFix = 4.0, kPartialRate = 3e6;

double split_cost(int ks, int M, int N) { return ks > 1 ? 2.0 * ks * static_cast<double>(N) * M * 4 / kPartialRate : 0.0; }

// Tiles and splits of the products that run together.  A product takes big
// tiles when its best estimate alone on the chip beats 128 x 128 tiles'
// throughput; the others share a launch and are cut into slices of at most
// `len` steps each, for the len with the least estimated time (the longest
// workgroup, or all of them over the CUs).
void plan_batch(const Item *it, int n, BPlan *out) {
  auto split = [](int steps, int ks, BPlan &p) {
    p.per = std::max(1, (steps + ks - 1) / ks);
    p.ksplit = std::max(1, (steps + p.per - 1) / p.per);
  };
  bool any_mid = false;
  for (int i = 0; i < n; ++i) {
    BPlan &p = out[i];
    p.nM = (it[i].M + 255) / 256;
    p.nN = (it[i].N + 255) / 256;
    const int64_t tiles = static_cast<int64_t>(p.nM) * p.nN;
    double best = 1e300;
    for (int ks = 1; ks <= 8 && ks * 8 <= std::max(8, it[i].steps); ++ks) {
      BPlan q{};
      split(it[i].steps, ks, q);
      const double rounds = static_cast<double>((tiles * q.ksplit + kCUs - 1) / kCUs);
      const double us = rounds * (q.per * kBigStep + kBigFix) + split_cost(q.ksplit, it[i].M, it[i].N) +
                        (q.ksplit > 1 ? kSumFix : 0.0);
      if (us < best) {
        best = us;
        p.per = q.per;
        p.ksplit = q.ksplit;
      }
    }
    const int mM = (it[i].M + 127) / 128, mN = (it[i].N + 127) / 128;
    p.big = !it[i].pair && best < static_cast<double>(mM) * mN * (it[i].steps * kMidPairStep + kMidFix) / (2 * kCUs) &&
            tiles * p.ksplit * 2 >= kCUs;
    if (!p.big) {
      p.nM = mM;
      p.nN = mN;
      any_mid = true;
    }
  }
  if (!any_mid) return;
  double best = 1e300;
  int best_len = 1 << 30;
  for (int len : {4, 6, 8, 12, 16, 24, 32, 48, 64, 96, 128, 1 << 20}) {
    double units = 0, work = 0, longest = 0, extra = 0;
    for (int pass = 0; pass < 2; ++pass) {
      const double step = pass && units > kCUs ? kMidPairStep : kMidStep;
      if (pass) work = longest = 0;
      for (int i = 0; i < n; ++i) {
        if (out[i].big) continue;
        BPlan q{};
        split(it[i].steps, std::clamp((it[i].steps + len - 1) / len, 1, 16), q);
        const double cnt = static_cast<double>(out[i].nM) * out[i].nN * q.ksplit, us = q.per * step + kMidFix;
        if (!pass) {
          units += cnt;
          extra += split_cost(q.ksplit, it[i].M, it[i].N);
          if (q.ksplit > 1 && extra < kSumFix) extra += kSumFix;
        } else {
          work += cnt * us;
          longest = std::max(longest, us);
        }
      }
    }
    const double slots = units > kCUs ? 2.0 * kCUs : kCUs;
    const double us = (units <= slots ? longest : std::max(longest, work / slots) + 0.5 * longest) + extra;
    if (us < best) {
      best = us;
      best_len = len;
    }
  }
  for (int i = 0; i < n; ++i)
    if (!out[i].big) split(it[i].steps, std::clamp((it[i].steps + best_len - 1) / best_len, 1, 16), out[i]);
}

int steps_of(int64_t len) { return static_cast<int>((len + kStep - 1) / kStep); }
int pad8(int n) { return (n + 7) & ~7; }
size_t pad256(size_t n) { return (n + 255) & ~size_t{255}; }

// Column slots of dy: every child's, then the tied v slot (k's rows again).
struct Slots {
  int n = 0, ldy = 0, ldd = 0;
  int child[kMaxChildren] = {}, from[kMaxChildren] = {}, start[kMaxChildren + 1] = {}, cols[kMaxChildren] = {};
  bool even = true;  // every slot already starts at a multiple of 8 of dy's rows
};

Slots slots_of(const CallDesc &c) {
  Slots s;
  auto add = [&](int child, int from, int cols) {
    s.child[s.n] = child;
    s.from[s.n] = from;
    s.cols[s.n] = cols;
    s.start[s.n] = s.ldd;
    s.ldd += pad8(cols);
    s.ldy = std::max(s.ldy, from + cols);
    if (from % 8 || cols % 8) s.even = false;
    ++s.n;
  };
  for (int i = 0; i < c.nchild; ++i) add(i, c.ch[i].y_off, c.ch[i].N);
  for (int i = 0; i < c.nchild; ++i)
    if (c.ch[i].dup_off >= 0) add(i, c.ch[i].dup_off, c.ch[i].N);
  s.start[s.n] = s.ldd;
  return s;
}

int slots_of_child(const Slots &s, int child) {
  int n = 0;
  for (int i = 0; i < s.n; ++i) n += s.child[i] == child;
  return n;
}

// The two batches of a call, planned as if every gradient were wanted (so that
// asking for fewer changes no bits): z and every g; then dx and every child's
// G, dU and dV.  A product of extent 0 (no rank) keeps its place.
struct Plans {
  BPlan z, g[kMaxChildren], dx, G[kMaxChildren], du[kMaxChildren], dv[kMaxChildren];
  bool few;     // dx (its plan) and every G in one pass
  size_t part;  // bytes of the larger batch's partials
};

// One pass over W0 for dx and G: few tokens, one dy slot per row of W0 (a tied
// v slot would need G summed over two), and a block worth another launch.
bool few_tokens(const CallDesc &c, const Slots &s, int T) {
  return T <= kFewPanels * kPanel && s.n == c.nchild && static_cast<int64_t>(c.Ntot) * c.K >= kFewBlock;
}

int few_panels(int T) { return T <= kPanel ? 1 : kFewPanels; }

// Slices of its rows: the fewest rounds of steps over the CUs.
void plan_few(int K, int steps, BPlan &p) {
  p = BPlan{};
  p.nM = (K + 127) / 128;
  p.nN = 1;
  int64_t best = INT64_MAX;
  for (int ks = 1; ks <= 32 && ks <= std::max(1, steps / 4); ++ks) {
    const int per = std::max(1, (steps + ks - 1) / ks), n = std::max(1, (steps + per - 1) / per);
    const int64_t cost = (static_cast<int64_t>(p.nM) * n + kCUs - 1) / kCUs * (per + 6);
    if (cost < best) {
      best = cost;
      p.per = per;
      p.ksplit = n;
    }
  }
}

Plans plans_of(const CallDesc &c, const Slots &s, int T) {
  Plans p{};
  Item it[kMaxProb];
  BPlan *to[kMaxProb], got[kMaxProb];
  int n = 0;
  auto add = [&](int M, int N, int steps, BPlan &dst, bool pair = false) {
    if (M == 0) return;
    it[n] = Item{M, N, steps, pair};
    to[n++] = &dst;
  };
  auto done = [&](size_t bytes) {
    plan_batch(it, n, got);
    for (int i = 0; i < n; ++i) {
      *to[i] = got[i];
      bytes += got[i].partial_bytes(it[i].M, it[i].N);
    }
    p.part = std::max(p.part, bytes);
    n = 0;
  };
  add(c.Rz, T, steps_of(c.K), p.z, true);
  for (int i = 0; i < c.nchild; ++i) add(c.ch[i].rpad, T, slots_of_child(s, i) * steps_of(c.ch[i].N), p.g[i], true);
  done(0);
  int dx_steps = 2 * steps_of(c.Rz);  // g's pair
  for (int i = 0; i < s.n; ++i) dx_steps += steps_of(s.cols[i]);
  p.few = few_tokens(c, s, T);
  if (p.few)
    plan_few(c.K, dx_steps, p.dx);
  else
    add(c.K, T, dx_steps, p.dx);
  for (int i = 0; i < c.nchild; ++i) {
    const int steps = slots_of_child(s, i) * steps_of(T);
    if (!p.few) add(c.K, c.ch[i].N, steps, p.G[i]);
    add(c.ch[i].rpad, c.ch[i].N, 2 * steps, p.du[i]);
    add(c.ch[i].rpad, c.K, 2 * steps_of(T), p.dv[i]);
  }
  done(p.few ? p.dx.partial_bytes(c.K, T) : 0);
  return p;
}

// Workspace: X bf16 [T][K], dy copies [T][ldd] x 2, z and g as pairs [T][2 Rz], the ds
// partial sums, and the K-split partials of a batch.
struct Offsets {
  size_t x, dyp, dys, z, g, dsp, dyt, xt, part, bytes;
};

Offsets offsets_of(const CallDesc &c, const Slots &s, const Plans &p, int T) {
  Offsets o{};
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t here = at;
    at += pad256(n);
    return here;
  };
  o.x = take(static_cast<size_t>(T) * c.K * 2);
  o.dyp = take(static_cast<size_t>(T) * s.ldd * 2);
  o.dys = take(static_cast<size_t>(T) * s.ldd * 2);
  o.z = take(static_cast<size_t>(T) * c.Rz * 4);
  o.g = take(static_cast<size_t>(T) * c.Rz * 4);
  o.dsp = take(static_cast<size_t>((c.K + 127) / 128) * 2 * c.Ntot * 4);
  const size_t few = p.few ? static_cast<size_t>(few_panels(T)) * kPanel * 2 : 0;
  o.dyt = take(s.ldd * few);
  o.xt = take(c.K * few);
  o.part = take(p.part);
  o.bytes = at;
  return o;
}

// Products that run together.
struct Batch {
  int n = 0;
  Prob p[kMaxProb];
  bool big[kMaxProb];
  const FewArgs *few = nullptr;  // dx and G in one pass
};

template <typename TL, auto KERN>
hipError_t launch_kernel(BwdArgs &a, hipStream_t stream) {
  const hipError_t e = ensure_lds<KERN>(TL::LDS);
  if (e != hipSuccess) return e;
  std::fill(a.unit0 + a.nprob, a.unit0 + kMaxProb, kNoUnit);
  hipLaunchKernelGGL(KERN, dim3(a.total), dim3(TL::NW * 64), TL::LDS, stream, a);
  return hipGetLastError();
}

template <bool BTR>
hipError_t launch_big(BwdArgs &a, hipStream_t stream) {
  return launch_kernel<Big<BTR>, product_kernel<Big<BTR>, true, BTR>>(a, stream);
}

template <typename TL>
hipError_t launch_few(const FewArgs &a, hipStream_t stream) {
  const hipError_t e = ensure_lds<few_kernel<TL>>(TL::RING);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(few_kernel<TL>, dim3(a.p.nM * a.p.ksplit), dim3(kFewWaves * 64), TL::RING, stream, a);
  return hipGetLastError();
}

void add_units(BwdArgs &a, const Prob &p) {
  a.unit0[a.nprob] = a.total;
  a.p[a.nprob++] = p;
  a.total += p.nM * p.nN * p.ksplit;
}

// The products of a batch -- big tiles by kind, then all others, the longest
// workgroups first -- and the launch that sums what they left.
hipError_t launch_batch(const Batch &b, hipStream_t stream) {
  hipError_t e;
  if (b.few) {
    e = b.few->p.N <= kPanel ? launch_few<FewTile<1>>(*b.few, stream) : launch_few<FewTile<kFewPanels>>(*b.few, stream);
    if (e != hipSuccess) return e;
  }
  for (int kind = kColsRows; kind <= kColsCols; ++kind) {  // (dx and G)
    BwdArgs a{};
    for (int i = 0; i < b.n; ++i)
      if (b.big[i] && b.p[i].kind == kind) add_units(a, b.p[i]);
    if (!a.nprob) continue;
    e = kind == kColsCols ? launch_big<true>(a, stream) : launch_big<false>(a, stream);
    if (e != hipSuccess) return e;
  }
  int order[kMaxProb], nmid = 0;
  for (int i = 0; i < b.n; ++i)
    if (!b.big[i]) order[nmid++] = i;
  std::stable_sort(order, order + nmid, [&](int x, int y) { return b.p[x].per > b.p[y].per; });
  if (nmid) {
    BwdArgs a{};
    for (int i = 0; i < nmid; ++i) add_units(a, b.p[order[i]]);
    e = a.total > kCUs ? launch_kernel<Mid2, products_kernel<Mid2>>(a, stream)
                       : launch_kernel<Mid4, products_kernel<Mid4>>(a, stream);
    if (e != hipSuccess) return e;
  }
  SumArgs a{};
  int blocks = 0;
  auto add_sum = [&](const Prob &p) {
    if (p.ksplit == 1 && !(p.mode == kWeight && p.ds)) return;
    a.first[a.nprob] = blocks;
    a.p[a.nprob++] = p;
    blocks += p.ksplit == 1       ? (p.N + 15) / 16
              : p.mode == kWeight ? p.N
                                  : static_cast<int>((static_cast<int64_t>(p.N) * (p.ldp / 4) + 255) / 256);
  };
  for (int i = 0; i < b.n; ++i) add_sum(b.p[i]);
  if (b.few) {
    Prob p = b.few->p;
    if (p.out) add_sum(p);
    p.mode = kWeight;  // ds, whose parts are not slices
    p.ksplit = 1;
    p.N = p.ldds;
    add_sum(p);
  }
  if (!a.nprob) return hipSuccess;
  std::fill(a.first + a.nprob, a.first + kMaxProb, kNoUnit);
  hipLaunchKernelGGL(sum_kernel, dim3(blocks), dim3(256), 0, stream, a);
  return hipGetLastError();
}

// Add a product to a batch; returns it for its segments and epilogue.  Its
// partials, sized for the planned extent Mp >= M (the padded rank), come from
// `part`.
Prob &add_product(Batch &b, const BPlan &pl, Kind kind, int M, int Mp, int N, uint16_t *out, int64_t ldo,
                  uint8_t *&part) {
  b.big[b.n] = pl.big;
  Prob &p = b.p[b.n++];
  p = Prob{};
  p.kind = kind;
  p.M = M;
  p.N = N;
  p.nM = pl.nM;
  p.nN = pl.nN;
  p.ksplit = pl.ksplit;
  p.per = pl.per;
  p.out = out;
  p.ldo = ldo;
  p.ldp = (Mp + 3) & ~3;
  p.P = reinterpret_cast<float *>(part);
  part += pl.partial_bytes(Mp, N);
  return p;
}

void add_seg(Prob &p, const uint16_t *A, int64_t lda, const uint16_t *B, int64_t ldb, int len) {
  p.seg[p.nseg++] = Seg{A, B, lda, ldb, len};
}

}  // namespace

size_t backward_workspace_bytes(const CallDesc &c, int T) {
  const Slots s = slots_of(c);
  return offsets_of(c, s, plans_of(c, s, T), T).bytes;
}

hipError_t launch_backward(const CallDesc &c, const CodedView &xc, const uint16_t *dy, const GradOut &o, void *ws_,
                           hipStream_t stream) {
  const int T = c.T, K = c.K;
  hipError_t e;
  bool want_u = false, want_v = false;
  for (int i = 0; i < c.nchild; ++i) {
    want_u |= o.du[i] && o.r[i];
    want_v |= o.dv[i] && o.r[i];
  }
  const bool want_w = o.ds || o.dw0, want_g = c.Rz > 0 && (o.dx || want_v);
  if (T == 0) {  // sums over no tokens
    if (o.ds && (e = launch_zero(o.ds, 2 * static_cast<int64_t>(c.Ntot), stream)) != hipSuccess) return e;
    if (o.dw0 && !o.accumulate && (e = launch_zero(o.dw0, 2 * static_cast<int64_t>(c.Ntot) * K, stream)) != hipSuccess)
      return e;
    for (int i = 0; i < c.nchild; ++i) {
      if ((e = launch_zero(o.du[i], static_cast<int64_t>(c.ch[i].N) * o.r[i], stream)) != hipSuccess) return e;
      if ((e = launch_zero(o.dv[i], static_cast<int64_t>(K) * o.r[i], stream)) != hipSuccess) return e;
    }
    return hipSuccess;
  }

  const Slots s = slots_of(c);
  const Plans pl = plans_of(c, s, T);
  uint8_t *ws = static_cast<uint8_t *>(ws_);
  const Offsets at = offsets_of(c, s, pl, T);
  uint16_t *X = reinterpret_cast<uint16_t *>(ws + at.x);
  uint16_t *z = reinterpret_cast<uint16_t *>(ws + at.z), *g = reinterpret_cast<uint16_t *>(ws + at.g);
  uint16_t *dys = reinterpret_cast<uint16_t *>(ws + at.dys);
  // dy as the products read it: itself where its slots lie on multiples of 8
  // columns and 16 bytes, else a copy where they do
  const bool direct = s.even && reinterpret_cast<uintptr_t>(dy) % 16 == 0;
  const uint16_t *dyp = direct ? dy : reinterpret_cast<const uint16_t *>(ws + at.dyp);
  const int64_t ldp = direct ? s.ldy : s.ldd;
  {
    PrepArgs a{};
    a.dy = dy;
    a.T = T;
    a.ldy = s.ldy;
    a.ldd = s.ldd;
    a.nslot = s.n;
    for (int i = 0; i < s.n; ++i) {
      a.start[i] = s.start[i];
      a.from[i] = s.from[i];
      a.n[i] = s.cols[i];
      a.s[i] = c.s + c.ch[s.child[i]].row_start;
    }
    a.start[s.n] = s.ldd;
    a.dyp = direct ? nullptr : reinterpret_cast<uint16_t *>(ws + at.dyp);
    a.dys = o.dx ? dys : nullptr;
    if (pl.few && want_w) {
      a.dyt = reinterpret_cast<uint16_t *>(ws + at.dyt);
      a.xt = reinterpret_cast<uint16_t *>(ws + at.xt);
    }
    // dy's columns are visited if any form of them is written
    a.dyb = a.dyp || a.dys || a.dyt ? (s.ldd / 8 + 255) / 256 : 0;
    a.xc = xc;
    a.K = K;
    a.X = X;
    const int xb = want_u || want_v || want_w ? (K / 8 + 255) / 256 : 0;
    a.cols = a.dyb + xb;
    if (a.cols > 0) {
      const int groups = ((a.xt ? few_panels(T) * kPanel : T) + kPrepT - 1) / kPrepT;
      hipLaunchKernelGGL(prepare_kernel, dim3(groups * a.cols), dim3(256), 0, stream, a);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
  }
  const int64_t ldz = 2 * static_cast<int64_t>(c.Rz);  // z and g: the values, then the remainders
  // rows of W0 from `row` on (null where no gradient asked for reads W0)
  auto block = [&](int row) { return c.W0 ? c.W0 + static_cast<int64_t>(row) * K : nullptr; };
  auto column = [&](int slot) { return dyp + (direct ? s.from[slot] : s.start[slot]); };
  {
    // z = X V and g = dy U
    uint8_t *part = ws + at.part;
    Batch b;
    if (want_u) {
      Prob &p = add_product(b, pl.z, kRowsRows, c.Rz, c.Rz, T, z, ldz, part);
      p.mode = kPair;
      p.lo = c.Rz;
      add_seg(p, c.Vt, K, X, K, K);
    }
    if (want_g)
      for (int i = 0; i < c.nchild; ++i) {
        const ChildDesc &ch = c.ch[i];
        if (!ch.rpad) continue;
        Prob &p = add_product(b, pl.g[i], kColsRows, ch.rpad, ch.rpad, T, g + ch.zoff, ldz, part);
        p.mode = kPair;
        p.lo = c.Rz;
        for (int j = 0; j < s.n; ++j)
          if (s.child[j] == i) add_seg(p, ch.U, ch.rpad, column(j), ldp, ch.N);
      }
    if ((e = launch_batch(b, stream)) != hipSuccess) return e;
  }
  uint8_t *part = ws + at.part;
  Batch b;
  auto dx_segments = [&](Prob &p) {  // dx = (dy (.) s) W0 + g V^T
    for (int j = 0; j < s.n; ++j)
      add_seg(p, block(c.ch[s.child[j]].row_start), K, dys + s.start[j], s.ldd, s.cols[j]);
    for (int lo = 0; lo < 2 && c.Rz > 0; ++lo) add_seg(p, c.Vt, K, g + lo * c.Rz, ldz, c.Rz);
  };
  FewArgs few{};
  if (pl.few && (o.dx || want_w)) {
    Batch one;
    few.p = add_product(one, pl.dx, kColsRows, K, K, T, o.dx, K, part);
    Prob &p = few.p;
    dx_segments(p);
    if (!o.dx) p.nseg = s.n;
    p.s = c.s;
    p.dw0 = o.dw0;
    p.accumulate = o.dw0 ? o.accumulate : 0;
    p.ds = o.ds;
    p.dsp = reinterpret_cast<float *>(ws + at.dsp);
    p.ldds = c.Ntot;
    few.nslot = s.n;
    for (int j = 0; j < s.n; ++j) {
      few.row[j] = c.ch[s.child[j]].row_start;
      few.dyt[j] = reinterpret_cast<const uint16_t *>(ws + at.dyt) + static_cast<int64_t>(s.start[j]) * kPanel;
    }
    few.dpanel = static_cast<int64_t>(s.ldd) * kPanel;
    few.xt = reinterpret_cast<const uint16_t *>(ws + at.xt);
    b.few = &few;
  } else if (o.dx) {
    dx_segments(add_product(b, pl.dx, kColsRows, K, K, T, o.dx, K, part));
  }
  for (int i = 0; i < c.nchild; ++i) {
    // G (dW0 and ds), dU and dV: contractions over the tokens
    const ChildDesc &ch = c.ch[i];
    auto add_tokens = [&](Prob &p, const uint16_t *A, int64_t lda) {
      for (int j = 0; j < s.n; ++j)
        if (s.child[j] == i) add_seg(p, A, lda, column(j), ldp, T);
    };
    if (want_w && !pl.few) {
      Prob &p = add_product(b, pl.G[i], kColsCols, K, K, ch.N, nullptr, 0, part);
      add_tokens(p, X, K);
      p.mode = kWeight;
      p.s = c.s + ch.row_start;
      p.W0 = block(ch.row_start);
      p.dw0 = o.dw0 ? o.dw0 + static_cast<int64_t>(ch.row_start) * K : nullptr;
      p.accumulate = o.dw0 ? o.accumulate : 0;
      p.ds = o.ds ? o.ds + ch.row_start : nullptr;
      p.dsp = reinterpret_cast<float *>(ws + at.dsp) + ch.row_start;
      p.ldds = c.Ntot;
    }
    if (o.du[i] && o.r[i]) {
      Prob &p = add_product(b, pl.du[i], kColsCols, o.r[i], ch.rpad, ch.N, o.du[i], o.r[i], part);
      for (int lo = 0; lo < 2; ++lo) add_tokens(p, z + ch.zoff + lo * c.Rz, ldz);
    }
    if (o.dv[i] && o.r[i]) {
      Prob &p = add_product(b, pl.dv[i], kColsCols, o.r[i], ch.rpad, K, o.dv[i], o.r[i], part);
      for (int lo = 0; lo < 2; ++lo) add_seg(p, g + ch.zoff + lo * c.Rz, ldz, X, K, T);
    }
  }
  return launch_batch(b, stream);
}

}  // namespace wl
