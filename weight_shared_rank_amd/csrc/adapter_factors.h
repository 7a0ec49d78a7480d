// The thin products of the adapters: z = c V^T X and g = c U^T dy of tiles of 64
// tokens, and what becomes of them: operands of the products that follow.
#pragma once

#include <type_traits>

#include "adapter_tiles.h"

namespace wl {

namespace {

constexpr int kM = 64;    // tokens of a tile
constexpr int kDeep = 4;  // stages under way
constexpr int kWaves = 8, kThreads = kWaves * 64;

// 8 codes and their scale byte as bf16, exact.
__device__ __forceinline__ u32x4 expand_codes(u32x2 v, uint8_t scale) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const float f = __uint_as_float(static_cast<uint32_t>(scale) << 23);
  u32x4 o;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(v[h]), false);
    const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(v[h]), true);
    o[2 * h] = pack_bf16(a[0] * f, a[1] * f);
    o[2 * h + 1] = pack_bf16(b[0] * f, b[1] * f);
  }
  return o;
}

// z and g summed over their slices, times c, in parts of bf16 in the operands' order.
// A piece is 64 lanes of 8 values:
//   transposed (for dU and dV): lane (r16, g) has rank 16 jt + r16 of positions
//     32 s + 8 g .. + 7 of the place: piece ((place * 2 + s) * RT + jt) * kParts + p
//   rows (for y and dx): lane (r16, g) has position 16 i + r16, ranks 32 ch + 8 g .. + 7 of
//     a child: piece ((place * 4 + i) * nchild * RC + child * RC + ch) * kParts + p
// with RT = R / 16, RC = r / 32 rounded up, p the part.
// Ranks past the slot's and positions behind the tile's tokens are zeros.
struct Factors {
  const float *scale;
  uint16_t *T[2];     // transposed z, g (null: not wanted)
  uint16_t *rows[2];  // rows
  int32_t RT, nchild, RC;
};

constexpr int kPieces = kParts * 512;  // elements of the pieces of a float's parts

// A lane's 8 values, their parts to as many pieces.
__device__ __forceinline__ void store_piece(uint16_t *to, int lane, const float (&v)[8]) {
  u32x2 o[2][kParts];
#pragma unroll
  for (int h = 0; h < 2; ++h) split4(f32x4{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]}, o[h]);
#pragma unroll
  for (int p = 0; p < kParts; ++p) *reinterpret_cast<u32x4 *>(to + p * 512 + lane * 8) = u32x4{o[0][p][0], o[0][p][1], o[1][p][0], o[1][p][1]};
}

// sum: [kM][pitch] floats of a place, column tile f of them is rank tile jt (of a
// child's) at column col of R.  A wave stores positions 32 s .. + 31 of it, in either
// order; with `last`, also the zeros of the rows piece's ranks behind it.
__device__ __forceinline__ void store_factors(const Factors &o, int which, int place0, int s, int col, int jt, bool last,
                                              const float *sum, int pitch, int f) {
  const int lane = threadIdx.x & 63, r16 = lane & 15, g = lane >> 4;
  float v[8];
  if (o.T[which]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = sum[(32 * s + 8 * g + k) * pitch + 16 * f + r16];
    store_piece(o.T[which] + ((static_cast<int64_t>(place0) * 2 + s) * o.RT + col / 16) * kPieces, lane, v);
  }
  if (o.rows[which]) {
    const int i = 2 * s + (g >> 1), child = (col / 16 - jt) / (o.RT / o.nchild), to = r16 + 16 * (2 * (jt & 1) + (g & 1));
    uint16_t *piece = o.rows[which] + ((static_cast<int64_t>(place0) * 4 + i) * o.nchild * o.RC + child * o.RC + jt / 2) * kPieces;
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = sum[(16 * i + r16) * pitch + 16 * f + 8 * (g & 1) + k];
    store_piece(piece, to, v);
    if (last && !(jt & 1)) {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = 0.f;
      store_piece(piece, to + 32, v);
    }
  }
}

// ---- z and g -------------------------------------------------------------------------
// P[slice][row][col] = sum over the slice of a thin operand's rows (V^T for z, U^T for
// g) times the tokens' x or dy.  A workgroup takes a tile, a slice and 16 NF columns; a
// stage of KS contraction values comes as rows, waits in registers while the kDeep - 1
// before it are used, and goes through LDS.  A wave multiplies two column tiles (one
// where there is no more) and 32 tokens over 32 values.
struct ProjectArgs {
  TileSource s;
  CodedView x;          // the checkpoint, or
  const uint16_t *xb;   // bf16 x [T][K]
  const uint16_t *vt;   // [n][nchild * r][K]
  const uint16_t *dy;   // [T][Ntot]
  const uint16_t *u;    // [n][Ntot][r]
  int32_t K, Ntot, nchild, N[kMaxChildren], n0[kMaxChildren];
  int32_t R;            // nchild * r
  int64_t rows;
  int32_t zgroups, zslices, zper;  // z: groups of NF column tiles, slices of K (0: no z), k of each
  int32_t ggroups, gslices, gper;  // g: groups of NF column tiles of a child, slices of N, n of each
  float *Pz, *Pg;       // [slices][rows][R]
  Factors out;
};

template <int NF>
struct Stage {
  static constexpr int KS = NF == 4 ? 64 : 128, SUBS = KS / 64, XB = SUBS * kM * 128;
  static constexpr int FP = NF == 4 ? 2 : 1, FR = NF == 1 ? 1 : 2, H = kWaves / (2 * FP);  // pairs of column tiles, tiles of a wave, waves along the contraction
  static constexpr int VB = SUBS * NF * 2048;                  // V^T: rows of 64 k
  static constexpr int UPITCH = 32 * (NF | 1), UB = KS * UPITCH;  // U: rows of 16 NF ranks
  static constexpr int BYTES = XB + (VB > UB ? VB : UB), SUMS = kWaves * FR * 2 * 1024;
  static constexpr int PITCH = 16 * NF + 1;  // of the sums, in floats
  static constexpr int LDS = 2 * BYTES > SUMS ? 2 * BYTES : SUMS;
  static_assert(kM * PITCH * 4 <= LDS, "the sums fit");
  static_assert(H * 32 == KS && XB == SUBS * kThreads * 16, "stage shape");
};

// Stages k0, k0 + KS, ... below k1 of a workgroup, kDeep under way: whole(d) loads the
// next whole stage, next() moves on by kDeep of them, last(k, d) loads a stage of which
// a part may lie past the end; put(d) and put_last(k, d) bring them to LDS, use(d)
// multiplies.
template <int KS, typename W, typename X, typename L, typename P, typename Q, typename U>
__device__ __forceinline__ void run_stages(int k0, int k1, W &&whole, X &&next, L &&last, P &&put, Q &&put_last, U &&use) {
  const int groups = (k1 - k0) / (KS * kDeep), kl = k0 + groups * KS * kDeep;
  if (groups > 0) {
#pragma unroll
    for (int d = 0; d < kDeep; ++d) whole(d);
    for (int i = 1; i < groups; ++i) {
      next();
#pragma unroll
      for (int d = 0; d < kDeep; ++d) {
        put(d);
        whole(d);
        use(d);
      }
    }
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      put(d);
      last(kl + d * KS, d);
      use(d);
    }
  } else {
#pragma unroll
    for (int d = 0; d < kDeep; ++d) last(kl + d * KS, d);
  }
#pragma unroll
  for (int d = 0; d < kDeep; ++d) {
    if (kl + d * KS >= k1) break;
    put_last(kl + d * KS, d);
    use(d);
  }
}

// The waves' sums along the contraction meet in LDS in wave order.  Column tile f of
// the workgroup is columns col(f) on of P's R, ranks rank0(f) on; with one slice alone
// they leave as finish_kernel would have them.
template <int NF, typename C, typename J>
__device__ __forceinline__ void store_sums(const ProjectArgs &a, const Tile &t, int which, int slice, const f32x4 (&acc)[Stage<NF>::FR][2],
                                           uint8_t *lds, int live, C &&col, J &&rank0) {
  using S = Stage<NF>;
  const int lane = threadIdx.x & 63, wave = keep(threadIdx.x >> 6), r16 = lane & 15, g = lane >> 4;
  const int fp = wave % S::FP, ip = wave / S::FP & 1, h = wave / (2 * S::FP);
  const bool one = (which ? a.gslices : a.zslices) == 1 && a.out.scale;
  f32x4 *part = reinterpret_cast<f32x4 *>(lds);  // [wave][FR][2][64]
  __syncthreads();
#pragma unroll
  for (int f = 0; f < S::FR; ++f)
#pragma unroll
    for (int i = 0; i < 2; ++i) part[((wave * S::FR + f) * 2 + i) * 64 + lane] = acc[f][i];
  __syncthreads();
  f32x4 v[S::FR][2];
  if (h == 0) {
#pragma unroll
    for (int f = 0; f < S::FR; ++f)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        v[f][i] = acc[f][i];
#pragma unroll
        for (int q = 1; q < S::H; ++q) v[f][i] += part[(((q * 2 * S::FP + wave) * S::FR + f) * 2 + i) * 64 + lane];
        const int tile = S::FR * fp + f, m = 32 * ip + 16 * i + r16;
        if (!one && tile < live && m < t.count)
          *reinterpret_cast<f32x4 *>((which ? a.Pg : a.Pz) + (slice * a.rows + static_cast<int64_t>(blockIdx.x) * kM + m) * a.R + col(tile) + g * 4) = v[f][i];
      }
  }
  if (!one) return;
  __syncthreads();
  float *sum = reinterpret_cast<float *>(lds);  // [kM][PITCH]
  if (h == 0) {
    const float scale = a.out.scale[t.slot];
#pragma unroll
    for (int f = 0; f < S::FR; ++f)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int tile = S::FR * fp + f, m = 32 * ip + 16 * i + r16;
          sum[m * S::PITCH + 16 * tile + 4 * g + k] = tile < live && m < t.count && rank0(tile) + 4 * g + k < t.rank ? v[f][i][k] * scale : 0.f;
        }
  }
  __syncthreads();
  const int f = wave >> 1, jt = rank0(f) / 16;
  if (wave < 2 * NF && f < live) store_factors(a.out, which, blockIdx.x, wave & 1, col(f), jt, jt == t.rank16 / 16 - 1, sum, S::PITCH, f);
}

template <int NF, bool CODED>
__device__ __forceinline__ void project_z(const ProjectArgs &a, const Tile &t, const int *tok, int unit, uint8_t *lds) {
  using S = Stage<NF>;
  constexpr int KS = S::KS, SUBS = S::SUBS;
  const int lane = threadIdx.x & 63, wave = keep(threadIdx.x >> 6), r16 = lane & 15, g = lane >> 4, K = a.K;
  const int f0 = unit % a.zgroups * NF, slice = unit / a.zgroups, per_child = t.rank16 / 16, live = a.nchild * per_child - f0;
  if (live <= 0) return;
  auto column = [&](int f) {  // tiles past the last repeat it
    const int v = f0 + min(f, live - 1);
    return v / per_child * a.s.r + v % per_child * 16;
  };
  const u32x4 zero{0u, 0u, 0u, 0u};
  const int chunk = threadIdx.x & 7, xrow = threadIdx.x >> 3;
  const int token = tok[xrow] < 0 ? tok[0] : tok[xrow];  // (columns without a token are not stored)
  const uint8_t *codes = a.x.codes + static_cast<int64_t>(token) * a.x.nb * kCodeBlock;
  const uint8_t *scales = a.x.scales + token;
  const uint16_t *xrows = a.xb + static_cast<int64_t>(token) * K;
  const int arow = (threadIdx.x >> 3) % (16 * NF), asub = threadIdx.x / (128 * NF) % SUBS;  // (NF 1: every piece twice)
  const uint16_t *a0 = a.vt + static_cast<int64_t>(t.slot) * a.R * K;
  const uint32_t arowb = static_cast<uint32_t>(column(arow >> 4) + (arow & 15)) * static_cast<uint32_t>(K) * 2u;
  const int ak = asub * 64 + chunk * 8;
  uint8_t *const xput = lds + xrow * 128 + (chunk ^ (xrow & 7)) * 16;
  uint8_t *const aput = lds + S::XB + (asub * 16 * NF + arow) * 128 + (chunk ^ (arow & 7)) * 16;
  const int fp = wave % S::FP, ip = wave / S::FP & 1, h = wave / (2 * S::FP), at = (((4 * h + g) & 7) ^ (r16 & 7)) * 16;
  const uint8_t *fa = lds + S::XB + ((h >> 1) * 16 * NF + 16 * S::FR * fp + r16) * 128 + at, *fx = lds + ((h >> 1) * kM + 32 * ip + r16) * 128 + at;
  f32x4 acc[S::FR][2];
#pragma unroll
  for (int f = 0; f < S::FR; ++f)
#pragma unroll
    for (int i = 0; i < 2; ++i) acc[f][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int k0 = slice * a.zper, k1 = min(K, k0 + a.zper);
  std::conditional_t<CODED, u32x2, u32x4> xv[kDeep][SUBS];
  uint8_t xs[kDeep];  // (a stage starts at a multiple of 64, SUBS 2: of 128: one block of codes)
  u32x4 av[kDeep];
  int k = k0;
  auto load = [&](int at_k, int d, bool whole) {
#pragma unroll
    for (int s = 0; s < SUBS; ++s) {
      const int kk = at_k + s * 64 + chunk * 8;
      if constexpr (CODED)
        xv[d][s] = *reinterpret_cast<const u32x2 *>(codes + (whole || kk < k1 ? kk : 0));
      else
        xv[d][s] = ld16(xrows + (whole || kk < k1 ? kk : 0));
    }
    if constexpr (CODED) xs[d] = scales[static_cast<int64_t>(whole || at_k < k1 ? at_k / kCodeBlock : 0) * a.x.ldsc];
    av[d] = whole ? ld16_at(a0 + at_k, arowb + ak * 2u) : ld16_at(a0, arowb + (at_k + ak < k1 ? (at_k + ak) * 2u : 0u));
  };
  auto put = [&](int at_k, int d, bool whole) {
    uint8_t *const to = lds + (d & 1) * S::BYTES;
#pragma unroll
    for (int s = 0; s < SUBS; ++s) {
      u32x4 v;
      if constexpr (CODED)
        v = expand_codes(xv[d][s], xs[d]);
      else
        v = xv[d][s];
      *reinterpret_cast<u32x4 *>(xput - lds + to + s * kM * 128) = whole || at_k + s * 64 + chunk * 8 < k1 ? v : zero;
    }
    *reinterpret_cast<u32x4 *>(aput - lds + to) = whole || at_k + ak < k1 ? av[d] : zero;
  };
  run_stages<KS>(
      k0, k1, [&](int d) { load(k + d * KS, d, true); }, [&] { k += KS * kDeep; }, [&](int at_k, int d) { load(at_k, d, false); },
      [&](int d) { put(0, d, true); }, [&](int at_k, int d) { put(at_k, d, false); },
      [&](int d) {
        wait_and_sync<63>();  // this stage is in LDS; loads stay under way
        const int buf = (d & 1) * S::BYTES;
        u32x4 x[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) x[i] = *reinterpret_cast<const u32x4 *>(fx + buf + i * 2048);
#pragma unroll
        for (int f = 0; f < S::FR; ++f) {
          const u32x4 v = *reinterpret_cast<const u32x4 *>(fa + buf + f * 2048);
#pragma unroll
          for (int i = 0; i < 2; ++i) acc[f][i] = mfma16x16x32(v, x[i], acc[f][i]);
        }
      });
  store_sums<NF>(a, t, 0, slice, acc, lds, live, column, [&](int f) { return (f0 + min(f, live - 1)) % per_child * 16; });
}

// ---- sums of the slices, where there are some -----------------------------------------------
struct FinishArgs {
  TileSource s;
  const float *P[2];     // z, g
  int32_t slices[2];     // below 2: nothing to do
  int32_t R;
  int64_t rows;
  Factors out;
};

__global__ __launch_bounds__(256) void finish_kernel(FinishArgs a) {
  constexpr int PITCH = 33;
  __shared__ int tok[kM];
  __shared__ float sum[kM * PITCH];
  Tile t;
  const int which = blockIdx.z;
  if (a.slices[which] < 2 || !get_tile<kM>(a.s, blockIdx.x, t, tok) || t.slot < 0) return;
  const int c = blockIdx.y / a.out.RC, ch = blockIdx.y % a.out.RC, j0 = ch * 32;  // ranks j0 .. + 31 of child c
  const float scale = a.out.scale[t.slot];
  {
    const int j = j0 + (threadIdx.x & 7) * 4;
    const bool in = j < a.s.r && j < t.rank16;
    const float *p = a.P[which] + (static_cast<int64_t>(blockIdx.x) * kM + (threadIdx.x >> 3)) * a.R + c * a.s.r + (in ? j : 0);
    const int64_t half = static_cast<int64_t>(32) * a.R, step = a.rows * a.R;
    f32x4 v[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
    if (in) {
#pragma unroll 4
      for (int s = 0; s < a.slices[which]; ++s) {
        v[0] += *reinterpret_cast<const f32x4 *>(p + s * step);
        v[1] += *reinterpret_cast<const f32x4 *>(p + s * step + half);
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int m = 32 * h + (threadIdx.x >> 3);
        sum[m * PITCH + (threadIdx.x & 7) * 4 + k] = m < t.count && in && j + k < t.rank ? v[h][k] * scale : 0.f;
      }
  }
  __syncthreads();
  const int w = threadIdx.x >> 6, jt = 2 * ch + (w & 1);
  if (16 * jt < a.s.r) store_factors(a.out, which, blockIdx.x, w >> 1, c * a.s.r + 16 * jt, jt, 16 * (jt + 1) == a.s.r, sum, PITCH, w & 1);
}

// Slices of a contraction: some workgroups for every CU, none below the shortest.
inline void cut_slices(int length, int stage, int shortest, int workgroups, int most, int &slices, int &per) {
  const int stages = (length + stage - 1) / stage;
  const int want = std::max(1, std::min({most, (3 * kCUs / 2 + workgroups - 1) / workgroups, stages / shortest}));
  per = (stages + want - 1) / want * stage;
  slices = (length + per - 1) / per;
}

}  // namespace

}  // namespace wl
