// Gradients of the low-rank adapters (adapters.hip) from an 8-bit checkpoint.
//
// With X the values of the checkpoint, dy the gradient of y and c the scale, per
// token z = c V^T X and g = c U^T dy, and
//   dx = base + V g,   dU_a = sum over the slot's tokens dy z^T,   dV_a^T = sum g X^T
// Launches, in tiles of 64 tokens: the grouping (not with few tokens); project_kernel, z
// and g, in float32 slices of the contraction where it is long; finish_kernel, their sums
// (with one slice of both, project_kernel's own end) in three parts of bf16, which
// hold all of a float32, each 16 x 32 piece of them stored as the 64 lanes' operand of a
// matrix instruction, so that the products load it as 1 KB; gradient_kernel, dx, dU and
// dV; with many tokens join_kernel, for slots whose tokens were cut for dU and dV.
//
// U (for g), V^T (for dx) and dy and X (for dU and dV) enter a product along
// their slow dimension.  They come from memory as rows, 16 bytes a lane, go through
// LDS, and are transposed on the way to the registers by ds_read_b64_tr_b16: 16 lanes
// read 4 rows of 16 elements, and lane l gets the 4 of column l.  Row 8 g + 4 h + i of
// 32 is kept at place 16 h + 4 g + i, so that the two reads of a fragment give lane
// group g its contraction values 8 g .. 8 g + 7 in order (what the other operand's 16
// bytes hold); with an odd multiple of 32 bytes from place to place, 8 neighbouring
// places lie in 8 different parts of the 256-byte bank period.
//
// Bound by memory: dy is read twice, for g and for dU, and everything else once.  As
// in the forward pass no load of a loop is conditional.  4096 tokens of 16 adapters
// through 31B gate|up, rank 32: 7 + 97 + 7 + 107 + 4 us; project_kernel reads 418 MB (4.3
// TB/s), gradient_kernel moves 560 MB (5.2 TB/s).  2048 tokens
// through 1B q|k|v: 6.4 + 9.4 + 11.7.  One pass over dy would hold dU of 64 columns and the
// child's ranks in a wave and write g of each 512 columns, 44 MB to and 44 from memory for the
// 352 it saves; not built.
#include <type_traits>

#include "adapter_factors.h"

namespace wl {

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// Place of a row (any number of 32s), in rows.
__device__ __forceinline__ int place(int row) {
  return (row & ~31) | ((row & 4) << 2) | ((row & 24) >> 1) | (row & 3);
}

// 16 columns of rows 32 b .. 32 b + 31: lane (r16, g) gets rows 8 g .. 8 g + 7 of
// column `r16` of those; at: byte offset of the four columns that lanes with
// these r16 & 3 read.
template <int PITCH>
__device__ __forceinline__ u32x4 read_transposed(const uint8_t *tile, int b, int at) {
  const int lane = threadIdx.x & 63, r16 = lane & 15, g = lane >> 4;
  const lds_u8 *p = (const lds_u8 *)tile + (32 * b + 4 * g + (r16 >> 2)) * PITCH + at;
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 16 * PITCH));
  const u32x2 x = __builtin_bit_cast(u32x2, lo), y = __builtin_bit_cast(u32x2, hi);
  return u32x4{x[0], x[1], y[0], y[1]};
}

// ---- g, and z beside it --------------------------------------------------------------
template <int NF>
__device__ __forceinline__ void project_g(const ProjectArgs &a, const Tile &t, const int *tok, int unit, uint8_t *lds) {
  using S = Stage<NF>;
  constexpr int KS = S::KS, SUBS = S::SUBS, LPR = 2 * NF;  // lanes of a row of U
  constexpr int UP = KS * LPR / kThreads ? KS * LPR / kThreads : 1;  // pieces of U of a thread (NF 1: every piece twice)
  const int lane = threadIdx.x & 63, wave = keep(threadIdx.x >> 6), r16 = lane & 15, g = lane >> 4;
  const int c = unit % a.nchild, j0 = unit / a.nchild % a.ggroups * NF * 16, slice = unit / a.nchild / a.ggroups;
  const int live = t.rank16 / 16 - j0 / 16, N = a.N[c], r = a.s.r;
  const int n0 = slice * a.gper, n1 = min(N, n0 + a.gper);
  if (live <= 0) return;
  const u32x4 zero{0u, 0u, 0u, 0u};
  const int chunk = threadIdx.x & 7, xrow = threadIdx.x >> 3;
  const uint16_t *dyrow = a.dy + static_cast<int64_t>(tok[xrow] < 0 ? tok[0] : tok[xrow]) * a.Ntot + a.n0[c] + chunk * 8;
  const uint16_t *U = a.u + (static_cast<int64_t>(t.slot) * a.Ntot + a.n0[c]) * r + j0;
  int urow[UP], ucol;
  uint32_t uoff[UP];
  uint8_t *uput[UP];
  ucol = threadIdx.x % LPR * 8;
#pragma unroll
  for (int i = 0; i < UP; ++i) {
    urow[i] = (i * kThreads + static_cast<int>(threadIdx.x)) / LPR % KS;
    uoff[i] = static_cast<uint32_t>(urow[i] * r + (j0 + ucol < r ? ucol : 0)) * 2u;  // (columns past the room: not stored)
    uput[i] = lds + S::XB + place(urow[i]) * S::UPITCH + ucol * 2;
  }
  uint8_t *const xput = lds + xrow * 128 + (chunk ^ (xrow & 7)) * 16;
  const int fp = wave % S::FP, ip = wave / S::FP & 1, h = wave / (2 * S::FP), at = (((4 * h + g) & 7) ^ (r16 & 7)) * 16;
  const uint8_t *fx = lds + ((h >> 1) * kM + 32 * ip + r16) * 128 + at;
  f32x4 acc[S::FR][2];
#pragma unroll
  for (int f = 0; f < S::FR; ++f)
#pragma unroll
    for (int i = 0; i < 2; ++i) acc[f][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  u32x4 xv[kDeep][SUBS], uv[kDeep][UP];
  int n = n0;
  run_stages<KS>(
      n0, max(n0, n1),
      [&](int d) {
#pragma unroll
        for (int s = 0; s < SUBS; ++s) xv[d][s] = ld16_any(dyrow + n + d * KS + s * 64);
#pragma unroll
        for (int i = 0; i < UP; ++i) uv[d][i] = ld16_at(U + static_cast<int64_t>(n + d * KS) * r, uoff[i]);
      },
      [&] { n += KS * kDeep; },
      [&](int at_n, int d) {  // the last stages: zeros past the slice
#pragma unroll
        for (int s = 0; s < SUBS; ++s) xv[d][s] = load_some(dyrow + at_n + s * 64, n1 - (at_n + s * 64 + chunk * 8));
#pragma unroll
        for (int i = 0; i < UP; ++i)
          uv[d][i] = at_n + urow[i] < n1 ? ld16_at(U + static_cast<int64_t>(at_n) * r, uoff[i]) : zero;
      },
      [&](int d) {
        const int buf = (d & 1) * S::BYTES;
#pragma unroll
        for (int s = 0; s < SUBS; ++s) *reinterpret_cast<u32x4 *>(xput + buf + s * kM * 128) = xv[d][s];
#pragma unroll
        for (int i = 0; i < UP; ++i) *reinterpret_cast<u32x4 *>(uput[i] + buf) = uv[d][i];
      },
      [&](int, int d) {
        const int buf = (d & 1) * S::BYTES;
#pragma unroll
        for (int s = 0; s < SUBS; ++s) *reinterpret_cast<u32x4 *>(xput + buf + s * kM * 128) = xv[d][s];
#pragma unroll
        for (int i = 0; i < UP; ++i) *reinterpret_cast<u32x4 *>(uput[i] + buf) = uv[d][i];
      },
      [&](int d) {
        wait_and_sync<63>();
        const int buf = (d & 1) * S::BYTES;
        u32x4 x[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) x[i] = *reinterpret_cast<const u32x4 *>(fx + buf + i * 2048);
#pragma unroll
        for (int f = 0; f < S::FR; ++f) {
          const u32x4 v = read_transposed<S::UPITCH>(lds + buf + S::XB, h, 32 * (S::FR * fp + f) + 8 * (r16 & 3));
#pragma unroll
          for (int i = 0; i < 2; ++i) acc[f][i] = mfma16x16x32(v, x[i], acc[f][i]);
        }
      });
  store_sums<NF>(a, t, 1, slice, acc, lds, live, [&](int f) { return c * r + j0 + 16 * f; }, [&](int f) { return j0 + 16 * f; });
}

template <int NF>
__global__ __launch_bounds__(kThreads, 4) void project_kernel(ProjectArgs a) {
  __shared__ int tok[kM];
  __shared__ __align__(16) uint8_t lds[Stage<NF>::LDS];
  Tile t;
  if (!get_tile<kM>(a.s, blockIdx.x, t, tok) || t.slot < 0) return;
  // the longer slices first (31B gate|up, g: 99 -> 96 us; 8192 -> 5376, z: 35 -> 31)
  const int units[2] = {a.zgroups * a.zslices, a.ggroups * a.nchild * a.gslices}, unit = blockIdx.y;
  const bool g_first = a.gper > a.zper;
  if (g_first ? unit < units[1] : unit >= units[0])
    project_g<NF>(a, t, tok, g_first ? unit : unit - units[0], lds);
  else
    project_z<NF, true>(a, t, tok, g_first ? unit - units[1] : unit, lds);
}

// ---- dx, dU, dV -----------------------------------------------------------------------------
constexpr int kGradWaves = 4, kPitch = 160, kPiece = 32 * kPitch;  // a wave's piece of LDS: 32 rows of 64 elements
constexpr int kOutPitch = 272;                                      // of sums: 16 rows of 64 floats
static_assert(16 * kOutPitch <= kPiece, "the sums fit the piece");

struct GradArgs {
  TileSource s;
  const int32_t *first, *count;  // per slot: first tile, tokens
  const int32_t *total;          // tiles, items, places
  const int4 *items;             // slot, cut, cuts, place among the slots' with more than one
  CodedView x;
  const uint16_t *vt, *dy;
  const uint16_t *zT, *gT, *grows;
  int32_t K, Ntot, nchild, N[kMaxChildren], n0[kMaxChildren];
  int32_t R, RC;
  const uint16_t *base;
  uint16_t *dx, *du, *dv;
  // the cuts of slots that have several: their sums, as the lanes hold them, KB by KB of
  // place * units + unit
  const int4 *joins;
  f32x4 *parts;
  int32_t units;  // a slot's column tiles times groups of ranks, dU's and then dV's
  // workgroups: dU and dV [items][groups of 16 JF ranks][column tiles of 64, or four of
  // them], then dx [K blocks of 256][half tiles]
  int32_t tiles, kblocks;
  int32_t jgroups;              // groups of ranks of a child
  int32_t ublock0[kMaxChildren + 1], vblocks;  // column tiles of the children's rows (running), of K
  int64_t blocks[3];            // of dU, dV, dx
};

// dx of 32 of a tile's tokens by 256 k, 64 a wave.  V^T rows of 32 ranks at a time and
// the sums pass through the wave's piece of LDS; base and dx move as 128 bytes a token.
__device__ __forceinline__ void dx_unit(const GradArgs &a, int64_t id, uint8_t *lds, int *tok) {
  Tile t;
  const int place0 = static_cast<int>(id % a.tiles), m0 = static_cast<int>(id / a.tiles % 2) * 32, kb = static_cast<int>(id / a.tiles / 2);
  if (!get_tile<kM>(a.s, place0, t, tok) || m0 >= t.count) return;
  const int lane = threadIdx.x & 63, wave = keep(threadIdx.x >> 6), r16 = lane & 15, g = lane >> 4;
  const int k0 = (kb * kGradWaves + wave) * 64, K = a.K;
  if (k0 >= K) return;
  uint8_t *const piece = lds + wave * kPiece;
  const int orow = lane >> 3, ocol = (lane & 7) * 8;
  const bool in = k0 + ocol < K;
  const u32x4 zero{0u, 0u, 0u, 0u};
  u32x4 b[2][2];
  int64_t at[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int token = tok[m0 + 16 * i + 8 * q + orow];
      at[i][q] = static_cast<int64_t>(token < 0 ? tok[0] : token) * K + (in ? k0 + ocol : 0);
      b[i][q] = ld16(a.base + at[i][q]);
    }
  if (t.slot >= 0) {
    f32x4 acc[4][2];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int chunks = (t.rank16 + 31) / 32, steps = a.nchild * chunks;
    const uint16_t *v0 = a.vt + static_cast<int64_t>(t.slot) * a.R * K;
    const uint16_t *g0 = a.grows + (static_cast<int64_t>(place0) * 4 + m0 / 16) * a.nchild * a.RC * kPieces;
    const uint32_t col = (in ? k0 + ocol : 0) * 2u;
    u32x4 vv[4], gv[2][kParts];
    auto load = [&](int step) {
      const int ch = step % chunks, c = step / chunks;
#pragma unroll
      for (int q = 0; q < 4; ++q)  // (rows past the rank repeat the last and are zeroed)
        vv[q] = ld16_at(v0, static_cast<uint32_t>(c * a.s.r + min(ch * 32 + q * 8 + orow, t.rank - 1)) * static_cast<uint32_t>(K) * 2u + col);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int p = 0; p < kParts; ++p) gv[i][p] = ld16_at(g0 + ((i * a.nchild * a.RC + c * a.RC + ch) * kParts + p) * 512, lane * 16u);
    };
    load(0);
    for (int step = 0; step < steps; ++step) {
      const int left = t.rank - step % chunks * 32;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<u32x4 *>(piece + place(q * 8 + orow) * kPitch + (lane & 7) * 16) = in && q * 8 + orow < left ? vv[q] : zero;
      u32x4 gg[2][kParts];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int p = 0; p < kParts; ++p) gg[i][p] = gv[i][p];
      load(min(step + 1, steps - 1));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const u32x4 v = read_transposed<kPitch>(piece, 0, 32 * j + 8 * (r16 & 3));
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int p = 0; p < kParts; ++p) acc[j][i] = mfma16x16x32(v, gg[i][p], acc[j][i]);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) *reinterpret_cast<f32x4 *>(piece + r16 * kOutPitch + (16 * j + 4 * g) * 4) = acc[j][i];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const f32x4 *o = reinterpret_cast<const f32x4 *>(piece + (8 * q + orow) * kOutPitch + ocol * 4);
        b[i][q] = add_8(b[i][q], o[0], o[1]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int q = 0; q < 2; ++q)
      if (in && m0 + 16 * i + 8 * q + orow < t.count) *reinterpret_cast<u32x4 *>(a.dx + at[i][q]) = b[i][q];
}

// Tokens of a slot.
struct Segment {
  int count, tile0, ntiles;  // tile0: its first tile of ntiles
  int from, stride, end;     // steps of 32 to take
  const int *list;           // or (FEW) the tokens, in LDS
};

// The sum over a slot's tokens for 64 columns of dy (dU) or of X (VGRAD: dV), by 16 JF
// ranks: 32 positions a step.  FULL: 64 columns exist.  ONCE: dy is read past the caches.
template <int JF, bool VGRAD, bool FEW, bool FULL, bool ONCE>
__device__ __forceinline__ void sum_tokens(const GradArgs &a, const Segment &seg, int c, int j0, int col0, int cols, uint8_t *piece,
                                           f32x4 (&acc)[4][JF]) {
  const int lane = threadIdx.x & 63, r16 = lane & 15, count = seg.count, from = seg.from, stride = seg.stride, steps = seg.end;
  const int RT = a.R / 16, col = col0 + (lane & 7) * 8;
  const u32x4 zero{0u, 0u, 0u, 0u};
  // the thin operand's pieces, from column tile (c r + j0) / 16 of z or g on
  const uint16_t *thin = (VGRAD ? a.gT : a.zT) + static_cast<int64_t>((c * a.s.r + j0) / 16) * kPieces;
  struct Rows {  // a step's place (halves of tiles), and the tokens of this lane's rows 8 q + lane / 8
    int half, token[4];
  };
  auto rows = [&](int step, Rows &o) {
    const bool real = step < steps;
    const int at = real ? step : from;
    if constexpr (FEW) {  // (a tile's place is its first token)
      o.half = keep(seg.list[(at >> 1) * kM]) * 2 + (at & 1);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int i = 32 * at + 8 * q + (lane >> 3), token = seg.list[min(i, count - 1)];
        o.token[q] = real && i < count ? token : -1;
      }
    } else {
      o.half = tile_place(seg.tile0 + (at >> 1), seg.ntiles) * 2 + (at & 1);
      const int32_t *p = a.s.perm + static_cast<int64_t>(o.half) * 32 + (lane >> 3);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int token = p[8 * q];
        o.token[q] = real ? token : -1;
      }
    }
  };
  struct Loaded {
    u32x4 w[VGRAD ? 1 : 4];
    u32x2 x[VGRAD ? 4 : 1];
    uint8_t s[VGRAD ? 4 : 1];
    u32x4 t[JF][kParts];
    uint32_t in;  // bits: the rows that are tokens
  };
  auto load = [&](const Rows &rw, Loaded &o) {
    o.in = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t row = max(rw.token[q], 0);  // (rows without a token are zeroed)
      o.in |= rw.token[q] >= 0 ? 1u << q : 0u;
      if constexpr (VGRAD) {
        const int kk = FULL || col < cols ? col : 0;
        o.x[q] = *reinterpret_cast<const u32x2 *>(a.x.codes + row * (a.x.nb * kCodeBlock) + kk);
        o.s[q] = a.x.scales[static_cast<int64_t>(kk / kCodeBlock) * a.x.ldsc + row];
      } else {
        const uint16_t *p = a.dy + row * a.Ntot + a.n0[c] + col;
        o.w[q] = !FULL ? load_some(p, cols - col) : ONCE ? ld16_any_once(p) : ld16_any(p);
      }
    }
    const uint16_t *p = thin + static_cast<int64_t>(rw.half) * RT * kPieces;
#pragma unroll
    for (int f = 0; f < JF; ++f) {
      const int ff = j0 + 16 * f < a.s.r ? f : 0;  // (not stored)
#pragma unroll
      for (int q = 0; q < kParts; ++q) o.t[f][q] = ld16_at(p + ff * kPieces + q * 512, lane * 16u);
    }
  };
  auto put = [&](const Loaded &o) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      u32x4 v;
      if constexpr (VGRAD)
        v = expand_codes(o.x[q], o.s[q]);
      else
        v = o.w[q];
      const bool in = (o.in >> q & 1) && (FULL || !VGRAD || col < cols);
      *reinterpret_cast<u32x4 *>(piece + place(q * 8 + (lane >> 3)) * kPitch + (lane & 7) * 16) = in ? v : zero;
    }
  };
  if (from >= steps) return;
  Rows next;
  Loaded l;
  rows(from, next);
  load(next, l);
  rows(from + stride, next);
  for (int step = from; step < steps; step += stride) {
    put(l);
    u32x4 t[JF][kParts];
#pragma unroll
    for (int f = 0; f < JF; ++f)
#pragma unroll
      for (int q = 0; q < kParts; ++q) t[f][q] = l.t[f][q];
    load(next, l);
    rows(step + 2 * stride, next);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // dV: 8 neighbouring k of a row end up in two accumulators of a lane
      const u32x4 w = read_transposed<kPitch>(piece, 0, VGRAD ? 64 * (i >> 1) + 16 * (r16 & 3) + 8 * (i & 1) : 32 * i + 8 * (r16 & 3));
#pragma unroll
      for (int f = 0; f < JF; ++f)
#pragma unroll
        for (int q = 0; q < kParts; ++q)
          acc[i][f] = VGRAD ? mfma16x16x32(w, t[f][q], acc[i][f]) : mfma16x16x32(t[f][q], w, acc[i][f]);
    }
  }
}

// Two neighbouring 16-column tiles (number `pair` of 64 from col0 on) of the 16 ranks from
// j on of child c to memory; zeros past the slot's rank, also where dy is not finite.
template <bool VGRAD>
__device__ __forceinline__ void store_sums_of(const GradArgs &a, int slot, int rank, int c, int j, int col0, int pair, f32x4 (&s)[2]) {
  const int lane = threadIdx.x & 63, r16 = lane & 15, g = lane >> 4, r = a.s.r;
  if (j >= r) return;
  if constexpr (VGRAD) {
    const int k = col0 + 32 * pair + 8 * g;
    if (j + r16 >= rank) s[0] = s[1] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (k < a.K)
      *reinterpret_cast<u32x4 *>(a.dv + (static_cast<int64_t>(slot) * a.R + c * r + j + r16) * a.K + k) =
          u32x4{pack_bf16(s[0][0], s[0][1]), pack_bf16(s[0][2], s[0][3]), pack_bf16(s[1][0], s[1][1]), pack_bf16(s[1][2], s[1][3])};
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int n = col0 + 16 * (2 * pair + h) + r16;
#pragma unroll
      for (int k = 0; k < 4; ++k) s[h][k] = j + 4 * g + k < rank ? s[h][k] : 0.f;
      if (n < a.N[c])
        *reinterpret_cast<u32x2 *>(a.du + (static_cast<int64_t>(slot) * a.Ntot + a.n0[c] + n) * r + j + 4 * g) =
            u32x2{pack_bf16(s[h][0], s[h][1]), pack_bf16(s[h][2], s[h][3])};
    }
  }
}

// Child of a column tile, which becomes the child's.
template <bool VGRAD>
__device__ __forceinline__ int child_of_tile(const GradArgs &a, int &ct) {
  int c = 0;
  if constexpr (VGRAD) {
    c = ct / a.vblocks;
    ct %= a.vblocks;
  } else {
#pragma unroll
    for (int i = 1; i < kMaxChildren; ++i)
      if (i < a.nchild && ct >= a.ublock0[i]) c = i;
    ct -= a.ublock0[c];
  }
  return c;
}

// WAYS 1: a wave has its own column tile; 4: the waves of a workgroup share one, a part of
// the tokens each.
template <int JF, bool VGRAD, int WAYS, bool FEW, bool ONCE>
__device__ __forceinline__ void weight_unit(const GradArgs &a, int64_t id, uint8_t *lds, int *list) {
  const int lane = threadIdx.x & 63, wave = keep(threadIdx.x >> 6);
  const int r = a.s.r;
  // column tiles fastest: the tiles of a slot run together
  const int blocks = VGRAD ? a.nchild * a.vblocks : a.ublock0[a.nchild], ctiles = (blocks * WAYS + 3) / 4;
  int ct = static_cast<int>(id % ctiles);
  const int64_t rest = id / ctiles;
  const int jg = static_cast<int>(rest % a.jgroups), j0 = jg * JF * 16, item = static_cast<int>(rest / a.jgroups);
  int slot = item, cut = 0, cuts = 1, place = 0;
  Segment seg{};
  if constexpr (FEW) {
    seg.count = keep(list_tokens(a.s, slot, list));
    seg.list = list;
  } else {
    if (item >= keep(a.total[1])) return;
    const int4 e = a.items[item];
    slot = keep(e.x);
    cut = keep(e.y);
    cuts = keep(e.z);
    place = keep(e.w);
    seg.count = keep(a.count[slot]);
    seg.tile0 = keep(a.first[slot]);
    seg.ntiles = keep(a.total[0]);
  }
  if constexpr (WAYS == 1) {
    ct = ct * 4 + wave;
    if (ct >= blocks) return;
  }
  const int unit = (VGRAD ? a.ublock0[a.nchild] * a.jgroups : 0) + jg * blocks + ct;
  const int steps = (seg.count + 31) / 32, per = (steps + cuts - 1) / cuts, lo = cut * per;
  seg.end = min(lo + per, steps);
  seg.from = WAYS == 1 ? lo : lo + wave;
  seg.stride = WAYS;
  const int c = child_of_tile<VGRAD>(a, ct);
  const int col0 = ct * 64, cols = VGRAD ? a.K : a.N[c];
  f32x4 acc[4][JF];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int f = 0; f < JF; ++f) acc[i][f] = f32x4{0.f, 0.f, 0.f, 0.f};
  uint8_t *const piece = lds + wave * kPiece;
  if (col0 + 64 <= cols)
    sum_tokens<JF, VGRAD, FEW, true, ONCE>(a, seg, c, j0, col0, cols, piece, acc);
  else
    sum_tokens<JF, VGRAD, FEW, false, ONCE>(a, seg, c, j0, col0, cols, piece, acc);
  const int rank = slot_rank(a.s.rank, r, slot);
  // a pair of column tiles of rank tile f: the cut's sums for join_kernel, or the gradient
  f32x4 *const parts = a.parts + (static_cast<int64_t>(place) * a.units + unit) * 4 * JF * 64 + lane;
  auto store = [&](f32x4 (&s)[2], int pair, int f) {
    if (cuts > 1) {
#pragma unroll
      for (int h = 0; h < 2; ++h) parts[((2 * pair + h) * JF + f) * 64] = s[h];
    } else {
      store_sums_of<VGRAD>(a, slot, rank, c, j0 + 16 * f, col0, pair, s);
    }
  };
  if constexpr (WAYS == 1) {
#pragma unroll
    for (int i = 0; i < 4; i += 2)
#pragma unroll
      for (int f = 0; f < JF; ++f) {
        f32x4 s[2] = {acc[i][f], acc[i + 1][f]};
        store(s, i / 2, f);
      }
  } else {
    // the waves' sums: two rank tiles at a time through LDS, in wave order
    constexpr int JC = JF < 2 ? JF : 2;
    f32x4 *part = reinterpret_cast<f32x4 *>(lds);  // [4 waves][4 column tiles][JC][64]
#pragma unroll
    for (int f0 = 0; f0 < JF; f0 += JC) {
      __syncthreads();
#pragma unroll
      for (int f = 0; f < JC; ++f)
#pragma unroll
        for (int i = 0; i < 4; ++i) part[((wave * 4 + i) * JC + f) * 64 + lane] = acc[i][f0 + f];
      __syncthreads();
      if ((wave >> 1) >= JC) continue;
      const int pair = wave & 1;
      f32x4 s[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x4 *p = part + ((2 * pair + h) * JC + (wave >> 1)) * 64 + lane;
        s[h] = p[0];
#pragma unroll
        for (int w = 1; w < kGradWaves; ++w) s[h] += p[w * 4 * JC * 64];
      }
      store(s, pair, f0 + (wave >> 1));
    }
  }
}

template <int JF, int WAYS, bool FEW, bool ONCE>
__global__ __launch_bounds__(kGradWaves * 64, JF == 4 ? 2 : 4) void gradient_kernel(GradArgs a) {
  constexpr int SUM = WAYS == 1 ? 0 : kGradWaves * 4 * (JF < 2 ? JF : 2) * 1024, PIECES = kGradWaves * kPiece;
  __shared__ int tok[FEW ? kLeaderT : kM];
  __shared__ __align__(16) uint8_t lds[SUM > PIECES ? SUM : PIECES];
  int64_t id = static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x;
  if (id < a.blocks[0]) return weight_unit<JF, false, WAYS, FEW, ONCE>(a, id, lds, tok);
  id -= a.blocks[0];
  if (id < a.blocks[1]) return weight_unit<JF, true, WAYS, FEW, ONCE>(a, id, lds, tok);
  id -= a.blocks[1];
  if (id < a.blocks[2]) dx_unit(a, id, lds, tok);
}

// The sums of a slot's cuts, in their order: a wave takes 32 columns of a unit and one
// rank tile.
template <int JF>
__global__ __launch_bounds__(256) void join_kernel(GradArgs a) {
  const int lane = threadIdx.x & 63, place = blockIdx.y;
  const int id = static_cast<int>(blockIdx.x) * 4 + keep(threadIdx.x >> 6), f = id / 2 % JF, pair = id & 1;
  int unit = id / (2 * JF);
  if (place >= keep(a.total[2]) || unit >= a.units) return;
  const int4 e = a.joins[place];
  const int slot = keep(e.x), cuts = keep(e.y);
  if (cuts == 0) return;
  const f32x4 *p = a.parts + ((static_cast<int64_t>(place) * a.units + unit) * 4 * JF + 2 * pair * JF + f) * 64 + lane;
  const int64_t next = static_cast<int64_t>(a.units) * 4 * JF * 64;
  f32x4 s[2] = {p[0], p[JF * 64]};
#pragma unroll 4
  for (int q = 1; q < cuts; ++q) {
    s[0] += p[q * next];
    s[1] += p[q * next + JF * 64];
  }
  const int rank = slot_rank(a.s.rank, a.s.r, slot), ublocks = a.ublock0[a.nchild];
  if (unit < ublocks * a.jgroups) {
    if (!a.du) return;
    int ct = unit % ublocks;
    const int j = (unit / ublocks * JF + f) * 16, c = child_of_tile<false>(a, ct);
    store_sums_of<false>(a, slot, rank, c, j, ct * 64, pair, s);
  } else {
    if (!a.dv) return;
    unit -= ublocks * a.jgroups;
    const int blocks = a.nchild * a.vblocks;
    int ct = unit % blocks;
    const int j = (unit / blocks * JF + f) * 16, c = child_of_tile<true>(a, ct);
    store_sums_of<true>(a, slot, rank, c, j, ct * 64, pair, s);
  }
}

__global__ __launch_bounds__(256) void fill_zero_16(u32x4 *p, int64_t n) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * 256)
    p[i] = u32x4{0u, 0u, 0u, 0u};
}

// ---- plan -----------------------------------------------------------------------------------
// dy, just read for g, is found in the caches while it is small; a larger one is read past
// them for dU, unless several groups of ranks read it (gradients of 31B gate|up with 16
// adapters of rank 16, through the caches and past them: 300 tokens, 26 MB, 51.6 and 53.6 us;
// 1000, 86 MB, 82.9 and 79.1; 4096, 352 MB, 193 and 186; of rank 128, two groups, 530 and 550).
constexpr int64_t kCachedDy = int64_t{64} << 20;

struct BackPlan {
  bool few;  // no grouping launch
  int tiles, NF, zgroups, zslices, zper, ggroups, gslices, gper, RC;
  int ublock0[kMaxChildren + 1], vblocks;
  int units, cut, places;  // of a slot; most steps of a cut; most cuts of slots that have several
  bool own;  // gradient_kernel's waves have column tiles of their own
  int64_t rows;
  size_t perm_at, slots_at, pz_at, pg_at, zt_at, gt_at, grows_at, items_at, joins_at, parts_at, bytes;
};

BackPlan make_back_plan(const AdapterPool &p, int T) {
  BackPlan q{};
  const int row_tiles = p.r / 16, R = p.nchild * p.r;
  q.NF = row_tiles >= 3 ? 4 : row_tiles;
  q.zgroups = (p.nchild * row_tiles + q.NF - 1) / q.NF;
  q.ggroups = (row_tiles + q.NF - 1) / q.NF;
  q.RC = (p.r + 31) / 32;
  int widest = 0;
  for (int c = 0; c < p.nchild; ++c) widest = std::max(widest, p.N[c]);
  const int stage = q.NF == 4 ? 64 : 128, busy = (T + kM - 1) / kM;
  // (one slice alone needs no finish_kernel: 77 tokens, 712 -> 1001: 21.1 -> 18.0 us; 2048
  // tokens through 1B q|k|v 31.2 -> 26.3)
  constexpr int kShortest = 2 * kDeep;
  cut_slices(p.K, stage, kShortest, busy * q.zgroups, 4, q.zslices, q.zper);
  cut_slices(widest, stage, kShortest, busy * q.ggroups * p.nchild, 8, q.gslices, q.gper);
  // Without the grouping a tile's place is its first token's, and workgroups at the other
  // places look and leave: pays while they are few (dx's for 77 tokens, 712 -> 1001, 480:
  // 17.4 -> 14.1 us; 8 of 4096 -> 4096, 256: 21.6 -> 19.1; 64 of them, 2048: 24.2 -> 25.1;
  // 256, 8192: 26.4 -> 39.6).
  const int64_t places = tile_places(T);
  q.few = T <= kLeaderT && places * 2 * ((p.K + 255) / 256) <= 4 * kCUs &&
          places * (q.zgroups * q.zslices + q.ggroups * p.nchild * q.gslices) <= 4 * kCUs;
  q.tiles = q.few ? tile_places(T) : tile_places(T / kM + std::min(p.n + 1, T));
  q.rows = static_cast<int64_t>(q.tiles) * kM;
  for (int c = 0; c < p.nchild; ++c) q.ublock0[c + 1] = q.ublock0[c] + (p.N[c] + 63) / 64;
  q.vblocks = (p.K + 63) / 64;
  q.units = q.ggroups * (q.ublock0[p.nchild] + p.nchild * q.vblocks);
  // Column tiles of their own save the waves the sums between them, where there are many
  // (16 adapters of 31B gate|up 134 -> 109 us, 32 of 8192 -> 5376 at rank 64 100 -> 75; but
  // 8 of 2048 -> 4096, 768 tiles, 12.2 -> 20.0, one of 31B gate|up, 840, 108 -> 133).
  q.own = static_cast<int64_t>(p.n) * q.units >= 4096;
  // How a call's tokens spread over the slots is not known here.  If one slot has them
  // all, its cuts are to keep 4 workgroups, or 16 waves, of a CU busy (3409 tokens in one
  // of 23 slots, 2 x 169 x 64 at rank 48: 85 -> 32 us; 8192 of one 1B q|k|v adapter 77 ->
  // 58; 4096 in one of 16 of 31B gate|up 288 -> 235, evenly spread 221).  Joining takes 4 us, cut
  // or not (2048 tokens of 8 1B q|k|v adapters 26.7 -> 31.8), so shorter calls go without (one of 8
  // slots of 4096 -> 2048 would gain 3 us from 2048 tokens; with own column tiles 1071
  // tokens in one of 34 slots 137 -> 85).  Cuts of 16 steps or 8, and of 24, 16 or 12 with
  // own tiles, differ by 10%.
  const int64_t steps = (T + 31) / 32;
  const int shortest = q.own ? 16 : 8, fewest = q.own ? 24 : 64;
  q.cut = static_cast<int>(std::max<int64_t>(shortest, steps * q.units / ((q.own ? 16 : 4) * kCUs)));
  if (steps <= fewest) q.cut = static_cast<int>(steps + 1);
  // Slots of more than `cut` steps: L of them have more than L cut of the steps + L there
  // can be, and s steps make at most s / cut + (cut - 1) / cut cuts.
  const int64_t L = steps / (q.cut - 1);
  q.places = steps > q.cut ? static_cast<int>((steps + L) / q.cut + L + 1) : 0;
  size_t at = align256(sizeof(int4) * q.tiles);  // the tiles come first
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align256(bytes);
    return here;
  };
  q.perm_at = take(sizeof(int32_t) * q.rows);
  q.slots_at = take(sizeof(int32_t) * (2 * static_cast<size_t>(p.n) + 3));
  q.items_at = take(sizeof(int4) * (static_cast<size_t>(p.n) + q.places));
  q.joins_at = take(sizeof(int4) * q.places);
  q.pz_at = take(sizeof(float) * q.zslices * q.rows * R);
  q.pg_at = take(sizeof(float) * q.gslices * q.rows * R);
  q.zt_at = take(kParts * sizeof(uint16_t) * q.rows * R);
  q.gt_at = take(kParts * sizeof(uint16_t) * q.rows * R);
  q.grows_at = take(kParts * sizeof(uint16_t) * q.rows * p.nchild * q.RC * 32);
  q.parts_at = take(size_t{4096} * q.NF * q.places * q.units);
  q.bytes = at;
  return q;
}

}  // namespace

size_t adapters_backward_workspace_bytes(const AdapterPool &p, int T) { return T > 0 ? make_back_plan(p, T).bytes : 256; }

hipError_t launch_adapters_backward(const AdapterPool &p, const CodedView &x, const uint16_t *dy, const int32_t *index, int T,
                                    const AdapterGrads &o, void *ws, hipStream_t stream) {
  if (T == 0) {
    if (!o.du && !o.dv) return hipSuccess;
    auto clear = [&](uint16_t *out, int64_t elements) {
      const int64_t n = elements / 8;
      if (out) fill_zero_16<<<static_cast<uint32_t>(std::min<int64_t>((n + 255) / 256, 8 * kCUs)), 256, 0, stream>>>(reinterpret_cast<u32x4 *>(out), n);
    };
    clear(o.du, static_cast<int64_t>(p.n) * p.Ntot * p.r);
    clear(o.dv, static_cast<int64_t>(p.n) * p.nchild * p.r * p.K);
    return hipGetLastError();
  }
  const BackPlan q = make_back_plan(p, T);
  const bool want_z = o.du, want_g = o.dx || o.dv;
  uint8_t *w = static_cast<uint8_t *>(ws);
  TileSource s{};
  s.index = index;
  s.rank = p.rank;
  s.T = T;
  s.n = p.n;
  s.r = p.r;
  s.copies = o.dx && o.dx != o.base;
  s.max_tiles = q.tiles;
  GroupArgs gr{};
  gr.s = s;
  gr.tiles = reinterpret_cast<int4 *>(w);
  gr.perm = reinterpret_cast<int32_t *>(w + q.perm_at);
  gr.first = reinterpret_cast<int32_t *>(w + q.slots_at);
  gr.count = gr.first + p.n;
  gr.total = gr.count + p.n;
  gr.items = reinterpret_cast<int4 *>(w + q.items_at);
  gr.cut = q.cut;
  gr.joins = reinterpret_cast<int4 *>(w + q.joins_at);
  hipError_t e = hipSuccess;
  if (!q.few) {
    if ((e = launch_group<kM>(gr, stream)) != hipSuccess) return e;
    s.tiles = gr.tiles;
    s.perm = gr.perm;
  }
  const int R = p.nchild * p.r;
  ProjectArgs a{};
  a.s = s;
  a.x = x;
  a.vt = p.vt;
  a.dy = dy;
  a.u = p.u;
  a.K = p.K;
  a.Ntot = p.Ntot;
  a.nchild = p.nchild;
  for (int c = 0, n0 = 0; c < p.nchild; ++c) {
    a.N[c] = p.N[c];
    a.n0[c] = n0;
    n0 += p.N[c];
  }
  a.R = R;
  a.rows = q.rows;
  a.zgroups = q.zgroups;
  a.zslices = want_z ? q.zslices : 0;
  a.zper = q.zper;
  a.ggroups = q.ggroups;
  a.gslices = want_g ? q.gslices : 0;
  a.gper = q.gper;
  a.Pz = reinterpret_cast<float *>(w + q.pz_at);
  a.Pg = reinterpret_cast<float *>(w + q.pg_at);
  a.out.scale = p.scale;
  a.out.T[0] = reinterpret_cast<uint16_t *>(w + q.zt_at);
  a.out.T[1] = o.dv ? reinterpret_cast<uint16_t *>(w + q.gt_at) : nullptr;
  a.out.rows[1] = o.dx ? reinterpret_cast<uint16_t *>(w + q.grows_at) : nullptr;
  a.out.RT = R / 16;
  a.out.nchild = p.nchild;
  a.out.RC = q.RC;
  const dim3 grid(q.tiles, a.zgroups * a.zslices + a.ggroups * p.nchild * a.gslices);
  if (q.NF == 1)
    project_kernel<1><<<grid, kThreads, 0, stream>>>(a);
  else if (q.NF == 2)
    project_kernel<2><<<grid, kThreads, 0, stream>>>(a);
  else
    project_kernel<4><<<grid, kThreads, 0, stream>>>(a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (a.zslices > 1 || a.gslices > 1) {
    FinishArgs f{};
    f.s = s;
    f.P[0] = a.Pz;
    f.P[1] = a.Pg;
    f.slices[0] = a.zslices;
    f.slices[1] = a.gslices;
    f.R = R;
    f.rows = q.rows;
    f.out = a.out;
    finish_kernel<<<dim3(q.tiles, p.nchild * q.RC, 2), 256, 0, stream>>>(f);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  GradArgs d{};
  d.s = s;
  d.first = gr.first;
  d.count = gr.count;
  d.total = gr.total;
  d.x = x;
  d.vt = p.vt;
  d.dy = dy;
  d.zT = a.out.T[0];
  d.gT = a.out.T[1];
  d.grows = a.out.rows[1];
  d.K = p.K;
  d.Ntot = p.Ntot;
  d.nchild = p.nchild;
  d.R = R;
  d.RC = q.RC;
  d.base = o.base;
  d.dx = o.dx;
  d.du = o.du;
  d.dv = o.dv;
  d.tiles = q.tiles;
  d.kblocks = (p.K + 255) / 256;
  d.vblocks = q.vblocks;
  for (int c = 0; c <= p.nchild; ++c) d.ublock0[c] = q.ublock0[c];
  for (int c = 0; c < p.nchild; ++c) {
    d.N[c] = a.N[c];
    d.n0[c] = a.n0[c];
  }
  d.jgroups = q.ggroups;
  d.items = gr.items;
  d.joins = gr.joins;
  d.parts = reinterpret_cast<f32x4 *>(w + q.parts_at);
  d.units = q.units;
  const int64_t items = p.n + (q.few ? 0 : q.places);
  auto blocks_of = [&](int tiles) { return items * d.jgroups * (q.own ? (tiles + 3) / 4 : tiles); };
  d.blocks[0] = o.du ? blocks_of(d.ublock0[p.nchild]) : 0;
  d.blocks[1] = o.dv ? blocks_of(p.nchild * d.vblocks) : 0;
  d.blocks[2] = o.dx ? static_cast<int64_t>(q.tiles) * 2 * d.kblocks : 0;
  const int64_t total = d.blocks[0] + d.blocks[1] + d.blocks[2];
  // (a launch holds fewer than 2^32 threads along x)
  constexpr int64_t kAcross = int64_t{1} << 20;
  const dim3 blocks(static_cast<uint32_t>(std::min(total, kAcross)), static_cast<uint32_t>((total + kAcross - 1) / kAcross));
  auto run = [&](auto jf) {
    constexpr int JF = decltype(jf)::value;
    if (q.few)
      q.own ? gradient_kernel<JF, 1, true, false><<<blocks, kGradWaves * 64, 0, stream>>>(d)
            : gradient_kernel<JF, 4, true, false><<<blocks, kGradWaves * 64, 0, stream>>>(d);
    else if (q.own && d.jgroups == 1 && static_cast<int64_t>(T) * p.Ntot * 2 > kCachedDy)
      gradient_kernel<JF, 1, false, true><<<blocks, kGradWaves * 64, 0, stream>>>(d);
    else
      q.own ? gradient_kernel<JF, 1, false, false><<<blocks, kGradWaves * 64, 0, stream>>>(d)
            : gradient_kernel<JF, 4, false, false><<<blocks, kGradWaves * 64, 0, stream>>>(d);
  };
  if (q.NF == 1)
    run(std::integral_constant<int, 1>{});
  else if (q.NF == 2)
    run(std::integral_constant<int, 2>{});
  else
    run(std::integral_constant<int, 4>{});
  if ((e = hipGetLastError()) != hipSuccess || q.places == 0 || d.blocks[0] + d.blocks[1] == 0) return e;
  const dim3 joins((q.units * 2 * q.NF + 3) / 4, q.places);
  if (q.NF == 1)
    join_kernel<1><<<joins, 256, 0, stream>>>(d);
  else if (q.NF == 2)
    join_kernel<2><<<joins, 256, 0, stream>>>(d);
  else
    join_kernel<4><<<joins, 256, 0, stream>>>(d);
  return hipGetLastError();
}

}  // namespace wl
