// Gradients of the low-rank adapters (adapters.hip) from an 8-bit checkpoint.
//
// With X the values of the checkpoint, dy the gradient of y and c the scale, per
// token z = c V^T X and g = c U^T dy, and
//   dx = base + V g,   dU_a = sum over the slot's tokens dy z^T,   dV_a^T = sum g X^T
// Launches: the grouping; project_kernel, z and g in float32 slices;
// finish_kernel, their sums as pairs of bf16 in the layouts the products read;
// gradient_kernel, dx, dU and dV.  Positions are the grouped order: tile * M + i.
//
// U (for g), V^T (for dx) and dy and X (for dU and dV) enter a product along
// their slow dimension.  They come from memory as they lie, 16 bytes a lane, go
// through a piece of LDS of the wave's own, and are transposed on the way to the
// registers by ds_read_b64_tr_b16: 16 lanes read 4 rows of 16 elements, and lane
// l gets the 4 of column l.  Row 8 g + 4 h + i of 32 is kept at place 16 h + 4 g + i,
// so that the two reads of a fragment give lane group g its contraction values
// 8 g .. 8 g + 7 in order (what the other operand's 16-byte loads hold), each
// from 16 places in a row; with an odd multiple of 32 bytes from place to place,
// 8 neighbouring places lie in 8 different parts of the 256-byte bank period.
#include "adapter_tiles.h"

namespace wl {

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;

// Place of a row (any number of 32s), in rows.
__device__ __forceinline__ int place(int row) {
  return (row & ~31) | ((row & 4) << 2) | ((row & 24) >> 1) | (row & 3);
}

// 16 columns of rows 32 b .. 32 b + 31: lane (r16, g) gets rows 8 g .. 8 g + 7 of
// column `r16` of those; at: byte offset of the four columns that lanes with
// these r16 & 3 read.
template <int PITCH>
__device__ __forceinline__ u32x4 read_transposed(const lds_u8 *tile, int b, int at) {
  const int lane = threadIdx.x & 63, r16 = lane & 15, g = lane >> 4;
  const lds_u8 *p = tile + (32 * b + 4 * g + (r16 >> 2)) * PITCH + at;
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 16 * PITCH));
  const u32x2 x = __builtin_bit_cast(u32x2, lo), y = __builtin_bit_cast(u32x2, hi);
  return u32x4{x[0], x[1], y[0], y[1]};
}

struct ProjectArgs {
  TileSource s;
  CodedView x;          // the checkpoint
  const uint16_t *vt;   // [n][nchild * r][K]
  const uint16_t *dy;   // [T][Ntot]
  const uint16_t *u;    // [n][Ntot][r]
  int32_t K, Ntot, nchild, N[kMaxChildren], n0[kMaxChildren];
  int32_t R;            // nchild * r
  int64_t rows;
  int32_t zgroups, zslices, zper;  // z: groups of NF row tiles, K slices, steps of each (zslices 0: no z)
  int32_t ggroups, gslices, gper;  // g: groups of NF row tiles of a child, slices of N, steps of each
  float *Pz, *Pg;       // [slices][rows][R]
};

constexpr int kM = 32, kMF = 2;  // tokens of a tile in the backward pass

// The waves' sums of a tile meet in LDS; wave 0 stores them.
template <int NF>
__device__ __forceinline__ void store_thin(const f32x4 (&acc)[NF][kMF], f32x4 *part, const int (&col)[NF], int live, int count,
                                           float *P, int64_t row0, int R) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r16 = lane & 15, g = lane >> 4;
  __syncthreads();
  if (wave > 0) {
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int i = 0; i < kMF; ++i) part[((wave - 1) * NF * kMF + f * kMF + i) * 64 + lane] = acc[f][i];
  }
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int i = 0; i < kMF; ++i) {
      f32x4 v = acc[f][i];
#pragma unroll
      for (int w = 0; w < 3; ++w) v += part[(w * NF * kMF + f * kMF + i) * 64 + lane];
      if (f < live && 16 * i + r16 < count) *reinterpret_cast<f32x4 *>(P + (row0 + 16 * i + r16) * R + col[f] + g * 4) = v;
    }
}

template <int NF>
__global__ __launch_bounds__(256) void project_kernel(ProjectArgs a) {
  constexpr int PITCH = 32 * (NF | 1), ROWS = NF == 8 ? 32 : 64, B = ROWS / 32;  // g: a wave's piece of U
  constexpr int PART = 3 * NF * kMF * 1024, PIECES = 4 * ROWS * PITCH;
  __shared__ int tok[kM];
  __shared__ __align__(16) uint8_t lds[PART > PIECES ? PART : PIECES];
  Tile t;
  if (!get_tile<kM>(a.s, blockIdx.x, t, tok) || t.slot < 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r16 = lane & 15, g = lane >> 4;
  const int per_child = t.rank16 / 16;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kM;
  const u32x4 zero{0u, 0u, 0u, 0u};
  f32x4 acc[NF][kMF];
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int i = 0; i < kMF; ++i) acc[f][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  int token[kMF], col[NF];
#pragma unroll
  for (int i = 0; i < kMF; ++i) token[i] = tok[16 * i + r16];
  int unit = blockIdx.y;
  const int zunits = a.zgroups * a.zslices;
  if (unit < zunits) {
    const int f0 = unit % a.zgroups * NF, slice = unit / a.zgroups, live = a.nchild * per_child - f0;
    if (live <= 0) return;
    const uint16_t *ar[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const int v = f0 + min(f, live - 1);
      col[f] = v / per_child * a.s.r + v % per_child * 16;
      ar[f] = a.vt + (static_cast<int64_t>(t.slot) * a.R + col[f] + r16) * a.K;
    }
    const int end = min((a.K + 63) / 64, (slice + 1) * a.zper);
    u32x4 xv[2][kMF][2], av[2][NF][2];
    auto load = [&](int step, u32x4(&xo)[kMF][2], u32x4(&ao)[NF][2]) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = step * 64 + g * 16 + h * 8;
        const bool in = step < end && k < a.K;
#pragma unroll
        for (int f = 0; f < NF; ++f) ao[f][h] = in ? ld16(ar[f] + k) : zero;
#pragma unroll
        for (int i = 0; i < kMF; ++i) xo[i][h] = in && token[i] >= 0 ? expand8(a.x, token[i], k) : zero;
      }
    };
    auto multiply = [&](const u32x4(&xo)[kMF][2], const u32x4(&ao)[NF][2]) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int f = 0; f < NF; ++f)
#pragma unroll
          for (int i = 0; i < kMF; ++i) acc[f][i] = mfma16x16x32(ao[f][h], xo[i][h], acc[f][i]);
    };
    int step = slice * a.zper + wave;
    load(step, xv[0], av[0]);
    for (; step < end; step += 8) {
      load(step + 4, xv[1], av[1]);
      multiply(xv[0], av[0]);
      load(step + 8, xv[0], av[0]);
      multiply(xv[1], av[1]);
    }
    store_thin<NF>(acc, reinterpret_cast<f32x4 *>(lds), col, live, t.count, a.Pz + slice * a.rows * a.R, row0, a.R);
    return;
  }
  unit -= zunits;
  const int c = unit % a.nchild, j0 = unit / a.nchild % a.ggroups * NF * 16, slice = unit / a.nchild / a.ggroups;
  const int live = per_child - j0 / 16, N = a.N[c];
  if (live <= 0) return;
#pragma unroll
  for (int f = 0; f < NF; ++f) col[f] = c * a.s.r + j0 + 16 * f;
  const uint16_t *U = a.u + (static_cast<int64_t>(t.slot) * a.Ntot + a.n0[c]) * a.s.r + j0;
  lds_u8 *piece = (lds_u8 *)lds + wave * (ROWS * PITCH);
  const int end = min((N + ROWS - 1) / ROWS, (slice + 1) * a.gper);
  constexpr int Q = ROWS * 2 * NF / 64;  // 16-byte loads of U a step and lane
  u32x4 uv[Q], dv[kMF][B];
  auto load = [&](int step) {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int v = q * 64 + lane, row = step * ROWS + v / (2 * NF), j = v % (2 * NF) * 8;
      uv[q] = step < end && row < N && j0 + j < a.s.r ? ld16(U + static_cast<int64_t>(row) * a.s.r + j) : zero;
    }
#pragma unroll
    for (int i = 0; i < kMF; ++i)
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const int n = step * ROWS + 32 * b + 8 * g;
        dv[i][b] = zero;
        if (step < end && token[i] >= 0 && n < N)
          dv[i][b] = load_some(a.dy + static_cast<int64_t>(token[i]) * a.Ntot + a.n0[c] + n, N - n);
      }
  };
  int step = slice * a.gper + wave;
  load(step);
  for (; step < end; step += 4) {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int v = q * 64 + lane;
      *(lds_u32x4 *)(piece + place(v / (2 * NF)) * PITCH + v % (2 * NF) * 16) = uv[q];
    }
    u32x4 d[kMF][B];
#pragma unroll
    for (int i = 0; i < kMF; ++i)
#pragma unroll
      for (int b = 0; b < B; ++b) d[i][b] = dv[i][b];
    load(step + 4);
#pragma unroll
    for (int b = 0; b < B; ++b)
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const u32x4 av = read_transposed<PITCH>(piece, b, 32 * f + 8 * (r16 & 3));
#pragma unroll
        for (int i = 0; i < kMF; ++i) acc[f][i] = mfma16x16x32(av, d[i][b], acc[f][i]);
      }
  }
  store_thin<NF>(acc, reinterpret_cast<f32x4 *>(lds), col, live, t.count, a.Pg + slice * a.rows * a.R, row0, a.R);
}

// z and g summed over their slices, times c, as pairs of bf16: transposed [2][R][rows]
// (dU, dV) and, for g, as rows [rows][2][R] (dx).  Columns past the slot's rank
// and positions behind the tile's tokens are zeros.
struct FinishArgs {
  TileSource s;
  const float *scale;
  const float *P[2];     // z, g
  int32_t slices[2];     // 0: not wanted
  int32_t R;
  int64_t rows;
  uint16_t *T[2];        // [2][R][rows]
  uint16_t *grows;       // [rows][2][R]
};

__global__ __launch_bounds__(256) void finish_kernel(FinishArgs a) {
  __shared__ int tok[kM];
  __shared__ uint16_t pair[2][32][kM + 2];
  Tile t;
  const int which = blockIdx.z;
  if (!a.slices[which] || !get_tile<kM>(a.s, blockIdx.x, t, tok) || t.slot < 0) return;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kM;
  const float scale = a.scale[t.slot];
  const int j0 = blockIdx.y * 32, l = threadIdx.x & 31;
  const int j = j0 + l;
#pragma unroll
  for (int m = threadIdx.x >> 5; m < kM; m += 8) {
    float v = 0.f;
    if (j < a.R && m < t.count && j % a.s.r < t.rank) {
      const float *p = a.P[which] + (row0 + m) * a.R + j;
      for (int s = 0; s < a.slices[which]; ++s) v += p[s * a.rows * a.R];
      v *= scale;
    }
    u32x2 hi2, lo2;
    split4(f32x4{v, 0.f, 0.f, 0.f}, hi2, lo2);
    const uint16_t h = static_cast<uint16_t>(hi2[0]), lo = static_cast<uint16_t>(lo2[0]);
    pair[0][l][m] = h;
    pair[1][l][m] = lo;
    if (which == 1 && a.grows && j < a.R) {
      a.grows[(row0 + m) * 2 * a.R + j] = h;
      a.grows[((row0 + m) * 2 + 1) * a.R + j] = lo;
    }
  }
  if (!a.T[which]) return;
  __syncthreads();
  // 32 rows of 32 positions, twice; 4 positions a thread
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = threadIdx.x >> 3, m = (threadIdx.x & 7) * 4;
    if (j0 + row >= a.R) continue;
    const uint16_t *p = &pair[i][row][m];
    *reinterpret_cast<u32x2 *>(a.T[which] + (static_cast<int64_t>(i) * a.R + j0 + row) * a.rows + row0 + m) =
        u32x2{p[0] | static_cast<uint32_t>(p[1]) << 16, p[2] | static_cast<uint32_t>(p[3]) << 16};
  }
}

struct GradArgs {
  TileSource s;
  const int32_t *first, *count;  // per slot: first tile, tokens
  const int32_t *total;          // tiles
  CodedView x;
  const uint16_t *vt, *dy;
  const uint16_t *zT, *gT, *grows;
  int32_t K, Ntot, nchild, N[kMaxChildren], n0[kMaxChildren];
  int32_t R;
  int64_t rows;
  const uint16_t *base;
  uint16_t *dx, *du, *dv;
  // workgroups: dx [tiles][K blocks of 256], then dU and dV [slots][column tiles
  // of 64][groups of 16 JF ranks]
  int32_t tiles, kblocks;
  int32_t jgroups;              // groups of ranks of a child
  int32_t ublock0[kMaxChildren + 1], vblocks;  // column tiles of the children's rows (running), of K
  int64_t units[3];             // dx, dU, dV
};

// dx of one tile: a wave takes 64 k.  V^T rows of 32 ranks at a time go through
// the wave's piece of LDS.
__device__ __forceinline__ void dx_unit(const GradArgs &a, int id, uint8_t *lds, int *tok) {
  Tile t;
  if (!get_tile<kM>(a.s, id / a.kblocks, t, tok)) return;
  constexpr int PITCH = 160;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r16 = lane & 15, g = lane >> 4;
  const int k0 = (id % a.kblocks * 4 + wave) * 64;
  if (k0 >= a.K) return;
  lds_u8 *piece = (lds_u8 *)lds + wave * (32 * PITCH);
  const u32x4 zero{0u, 0u, 0u, 0u};
  u32x4 b[kMF][2];
  int64_t at[kMF];
#pragma unroll
  for (int i = 0; i < kMF; ++i) {
    const int token = tok[16 * i + r16];
    at[i] = token < 0 ? -1 : static_cast<int64_t>(token) * a.K + k0 + 8 * g;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      b[i][h] = token >= 0 && k0 + 32 * h + 8 * g < a.K ? ld16(a.base + at[i] + 32 * h) : zero;
  }
  if (t.slot >= 0) {
    f32x4 acc[4][kMF];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < kMF; ++i) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int64_t row0 = static_cast<int64_t>(id / a.kblocks) * kM;
    const int chunks = (t.rank16 + 31) / 32, steps = a.nchild * chunks;
    u32x4 vv[4], gv[kMF][2];
    auto load = [&](int step) {
      const int j0 = step % chunks * 32, c0 = step / chunks * a.s.r;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int row = q * 8 + (lane >> 3), k = k0 + (lane & 7) * 8;
        vv[q] = step < steps && j0 + row < t.rank && k < a.K
                    ? ld16(a.vt + (static_cast<int64_t>(t.slot) * a.R + c0 + j0 + row) * a.K + k) : zero;
      }
#pragma unroll
      for (int i = 0; i < kMF; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          gv[i][h] = step < steps && j0 + 8 * g < t.rank16
                         ? ld16(a.grows + ((row0 + 16 * i + r16) * 2 + h) * a.R + c0 + j0 + 8 * g) : zero;
    };
    load(0);
    for (int step = 0; step < steps; ++step) {
#pragma unroll
      for (int q = 0; q < 4; ++q) *(lds_u32x4 *)(piece + place(q * 8 + (lane >> 3)) * PITCH + (lane & 7) * 16) = vv[q];
      u32x4 gg[kMF][2];
#pragma unroll
      for (int i = 0; i < kMF; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) gg[i][h] = gv[i][h];
      load(step + 1);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const u32x4 av = read_transposed<PITCH>(piece, 0, 64 * (j >> 1) + 16 * (r16 & 3) + 8 * (j & 1));
#pragma unroll
        for (int i = 0; i < kMF; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) acc[j][i] = mfma16x16x32(av, gg[i][h], acc[j][i]);
      }
    }
#pragma unroll
    for (int i = 0; i < kMF; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) b[i][h] = add_8(b[i][h], acc[2 * h][i], acc[2 * h + 1][i]);
  }
#pragma unroll
  for (int i = 0; i < kMF; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (at[i] >= 0 && k0 + 32 * h + 8 * g < a.K) *reinterpret_cast<u32x4 *>(a.dx + at[i] + 32 * h) = b[i][h];
}

// 64 columns of dy (VGRAD false: dU) or of X (dV) by 16 JF ranks of one slot: the
// sum over its tokens, 32 at a time, taken in turn by the four waves.
template <int JF, bool VGRAD>
__device__ __forceinline__ void weight_unit(const GradArgs &a, int64_t id, uint8_t *lds) {
  constexpr int PITCH = 160;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r16 = lane & 15, g = lane >> 4;
  const int r = a.s.r;
  // column tiles fastest: the tiles of a slot run together
  const int ctiles = VGRAD ? a.nchild * a.vblocks : a.ublock0[a.nchild];
  int ct = static_cast<int>(id % ctiles);
  const int64_t rest = id / ctiles;
  const int j0 = static_cast<int>(rest % a.jgroups) * JF * 16, slot = static_cast<int>(rest / a.jgroups);
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
  const int col0 = ct * 64, cols = VGRAD ? a.K : a.N[c];
  const int count = a.count[slot];
  const int tile0 = a.first[slot], ntiles = *a.total;
  lds_u8 *piece = (lds_u8 *)lds + wave * (32 * PITCH);
  const u32x4 zero{0u, 0u, 0u, 0u};
  // the thin operand, from column c * r + j0 of z (dU) or g (dV) on
  const uint16_t *thin = (VGRAD ? a.gT : a.zT) + (static_cast<int64_t>(c) * r + j0) * a.rows;
  const int64_t lo = static_cast<int64_t>(a.R) * a.rows;
  f32x4 acc[4][JF];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int f = 0; f < JF; ++f) acc[i][f] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int steps = (count + 31) / 32;
  u32x4 wv[4], tv[JF][2];
  int token[4];  // of the step after the one in wv
  auto tokens = [&](int step) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      token[q] = step < steps ? a.s.perm[static_cast<int64_t>(tile_place(tile0 + step, ntiles)) * kM + q * 8 + (lane >> 3)] : -1;
  };
  auto load = [&](int step) {
    const int k = col0 + (lane & 7) * 8;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      wv[q] = zero;
      if (token[q] >= 0 && k < cols) {
        if constexpr (VGRAD)
          wv[q] = expand8(a.x, token[q], k);
        else
          wv[q] = load_some(a.dy + static_cast<int64_t>(token[q]) * a.Ntot + a.n0[c] + k, cols - k);
      }
    }
#pragma unroll
    for (int f = 0; f < JF; ++f)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        tv[f][h] = step < steps && j0 + 16 * f < r
                       ? ld16(thin + h * lo + (16 * f + r16) * a.rows + static_cast<int64_t>(tile_place(tile0 + step, ntiles)) * kM + 8 * g) : zero;
  };
  tokens(wave);
  load(wave);
  tokens(wave + 4);
  for (int step = wave; step < steps; step += 4) {
#pragma unroll
    for (int q = 0; q < 4; ++q) *(lds_u32x4 *)(piece + place(q * 8 + (lane >> 3)) * PITCH + (lane & 7) * 16) = wv[q];
    u32x4 tt[JF][2];
#pragma unroll
    for (int f = 0; f < JF; ++f)
#pragma unroll
      for (int h = 0; h < 2; ++h) tt[f][h] = tv[f][h];
    load(step + 4);
    tokens(step + 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // dV: 8 neighbouring k of a row end up in two accumulators of a lane
      const u32x4 w = read_transposed<PITCH>(piece, 0, VGRAD ? 64 * (i >> 1) + 16 * (r16 & 3) + 8 * (i & 1) : 32 * i + 8 * (r16 & 3));
#pragma unroll
      for (int f = 0; f < JF; ++f)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          acc[i][f] = VGRAD ? mfma16x16x32(w, tt[f][h], acc[i][f]) : mfma16x16x32(tt[f][h], w, acc[i][f]);
    }
  }
  // the waves' sums: two rank tiles at a time through LDS, in wave order
  constexpr int JC = JF < 2 ? JF : 2;
  f32x4 *part = reinterpret_cast<f32x4 *>(lds);  // [4 waves][4 column tiles][JC][64]
  for (int f0 = 0; f0 < JF; f0 += JC) {
    __syncthreads();
#pragma unroll
    for (int f = 0; f < JF; ++f)
      if (f >= f0 && f < f0 + JC)
#pragma unroll
        for (int i = 0; i < 4; ++i) part[((wave * 4 + i) * JC + f - f0) * 64 + lane] = acc[i][f];
    __syncthreads();
    const int f = f0 + (wave >> 1);
    if ((wave >> 1) >= JC || j0 + 16 * f >= r) continue;
    f32x4 s[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f32x4 *p = part + ((2 * (wave & 1) + h) * JC + (wave >> 1)) * 64 + lane;
      s[h] = p[0];
#pragma unroll
      for (int w = 1; w < 4; ++w) s[h] += p[w * 4 * JC * 64];
    }
    if constexpr (VGRAD) {
      const int k = col0 + 32 * (wave & 1) + 8 * g, j = c * r + j0 + 16 * f + r16;
      if (k < a.K)
        *reinterpret_cast<u32x4 *>(a.dv + (static_cast<int64_t>(slot) * a.R + j) * a.K + k) =
            u32x4{pack_bf16(s[0][0], s[0][1]), pack_bf16(s[0][2], s[0][3]), pack_bf16(s[1][0], s[1][1]), pack_bf16(s[1][2], s[1][3])};
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int n = col0 + 16 * (2 * (wave & 1) + h) + r16;
        if (n < cols)
          *reinterpret_cast<u32x2 *>(a.du + (static_cast<int64_t>(slot) * a.Ntot + a.n0[c] + n) * r + j0 + 16 * f + 4 * g) =
              u32x2{pack_bf16(s[h][0], s[h][1]), pack_bf16(s[h][2], s[h][3])};
      }
    }
  }
}

template <int JF>
__global__ __launch_bounds__(256) void gradient_kernel(GradArgs a) {
  constexpr int SUM = 4 * 4 * (JF < 2 ? JF : 2) * 1024, PIECES = 4 * 32 * 160;
  __shared__ int tok[kM];
  __shared__ __align__(16) uint8_t lds[SUM > PIECES ? SUM : PIECES];
  int64_t id = static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x;
  if (id >= a.units[0] + a.units[1] + a.units[2]) return;
  if (id < a.units[0]) return dx_unit(a, static_cast<int>(id), lds, tok);
  id -= a.units[0];
  if (id < a.units[1]) return weight_unit<JF, false>(a, id, lds);
  weight_unit<JF, true>(a, id - a.units[1], lds);
}

__global__ __launch_bounds__(256) void fill_zero_16(u32x4 *p, int64_t n) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * 256)
    p[i] = u32x4{0u, 0u, 0u, 0u};
}

struct BackPlan {
  int tiles, NF, zgroups, zslices, zper, ggroups, gslices, gper;
  int64_t rows;
  size_t perm_at, slots_at, pz_at, pg_at, zt_at, gt_at, grows_at, bytes;
};

BackPlan make_back_plan(const AdapterPool &p, int T) {
  BackPlan q{};
  q.tiles = tile_places(T / kM + std::min(p.n + 1, T));
  q.rows = static_cast<int64_t>(q.tiles) * kM;
  const int row_tiles = p.r / 16, R = p.nchild * p.r;
  q.NF = row_tiles >= 8 ? 8 : row_tiles >= 3 ? 4 : row_tiles;
  q.zgroups = (p.nchild * row_tiles + q.NF - 1) / q.NF;
  q.ggroups = (row_tiles + q.NF - 1) / q.NF;
  int widest = 0;
  for (int c = 0; c < p.nchild; ++c) widest = std::max(widest, p.N[c]);
  const int zsteps = (p.K + 63) / 64, rows = q.NF == 8 ? 32 : 64, gsteps = (widest + rows - 1) / rows;
  const int busy = (T + kM - 1) / kM;
  auto cut = [&](int steps, int workgroups, int &slices, int &per) {
    const int want = std::min({8, (4 * kCUs + workgroups - 1) / workgroups, (steps + 3) / 4});
    per = (steps + want - 1) / want;
    slices = (steps + per - 1) / per;
  };
  cut(zsteps, busy * q.zgroups, q.zslices, q.zper);
  cut(gsteps, busy * q.ggroups * p.nchild, q.gslices, q.gper);
  size_t at = align256(sizeof(int4) * q.tiles);  // the tiles come first
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align256(bytes);
    return here;
  };
  q.perm_at = take(sizeof(int32_t) * q.rows);
  q.slots_at = take(sizeof(int32_t) * (2 * static_cast<size_t>(p.n) + 1));
  q.pz_at = take(sizeof(float) * q.zslices * q.rows * R);
  q.pg_at = take(sizeof(float) * q.gslices * q.rows * R);
  q.zt_at = take(2 * sizeof(uint16_t) * q.rows * R);
  q.gt_at = take(2 * sizeof(uint16_t) * q.rows * R);
  q.grows_at = take(2 * sizeof(uint16_t) * q.rows * R);
  q.bytes = at;
  return q;
}

}  // namespace

size_t adapters_backward_workspace_bytes(const AdapterPool &p, int T) { return T > 0 ? make_back_plan(p, T).bytes : 256; }

hipError_t launch_adapters_backward(const AdapterPool &p, const CodedView &x, const uint16_t *dy, const int32_t *index, int T,
                                    const AdapterGrads &o, void *ws, hipStream_t stream) {
  const size_t ub = static_cast<size_t>(p.n) * p.Ntot * p.r * 2, vb = static_cast<size_t>(p.n) * p.nchild * p.r * p.K * 2;
  if (T == 0) {
    if (!o.du && !o.dv) return hipSuccess;
    auto clear = [&](uint16_t *out, size_t bytes) {
      const int64_t n = static_cast<int64_t>(bytes / 16);
      if (out) fill_zero_16<<<static_cast<uint32_t>(std::min<int64_t>((n + 255) / 256, 8 * kCUs)), 256, 0, stream>>>(reinterpret_cast<u32x4 *>(out), n);
    };
    clear(o.du, ub);
    clear(o.dv, vb);
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
  group_kernel<kM><<<group_workgroups(p.n), kGroupWaves * 64, 0, stream>>>(gr);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  s.tiles = gr.tiles;
  s.perm = gr.perm;
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
  const dim3 grid(q.tiles, a.zgroups * a.zslices + a.ggroups * p.nchild * a.gslices);
  switch (q.NF) {
    case 1: project_kernel<1><<<grid, 256, 0, stream>>>(a); break;
    case 2: project_kernel<2><<<grid, 256, 0, stream>>>(a); break;
    case 4: project_kernel<4><<<grid, 256, 0, stream>>>(a); break;
    default: project_kernel<8><<<grid, 256, 0, stream>>>(a); break;
  }
  if ((e = hipGetLastError()) != hipSuccess) return e;
  FinishArgs f{};
  f.s = s;
  f.scale = p.scale;
  f.P[0] = a.Pz;
  f.P[1] = a.Pg;
  f.slices[0] = a.zslices;
  f.slices[1] = a.gslices;
  f.R = R;
  f.rows = q.rows;
  f.T[0] = reinterpret_cast<uint16_t *>(w + q.zt_at);
  f.T[1] = o.dv ? reinterpret_cast<uint16_t *>(w + q.gt_at) : nullptr;
  f.grows = o.dx ? reinterpret_cast<uint16_t *>(w + q.grows_at) : nullptr;
  finish_kernel<<<dim3(q.tiles, (R + 31) / 32, 2), 256, 0, stream>>>(f);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  GradArgs d{};
  d.s = s;
  d.first = gr.first;
  d.count = gr.count;
  d.total = gr.total;
  d.x = x;
  d.vt = p.vt;
  d.dy = dy;
  d.zT = f.T[0];
  d.gT = reinterpret_cast<uint16_t *>(w + q.gt_at);
  d.grows = f.grows;
  d.K = p.K;
  d.Ntot = p.Ntot;
  d.nchild = p.nchild;
  d.R = R;
  d.rows = q.rows;
  d.base = o.base;
  d.dx = o.dx;
  d.du = o.du;
  d.dv = o.dv;
  d.tiles = q.tiles;
  d.kblocks = (p.K + 255) / 256;
  d.vblocks = (p.K + 63) / 64;
  for (int c = 0; c < p.nchild; ++c) {
    d.N[c] = a.N[c];
    d.n0[c] = a.n0[c];
    d.ublock0[c + 1] = d.ublock0[c] + (p.N[c] + 63) / 64;
  }
  const int JF = q.NF;
  d.jgroups = q.ggroups;
  d.units[0] = o.dx ? static_cast<int64_t>(q.tiles) * d.kblocks : 0;
  d.units[1] = o.du ? static_cast<int64_t>(p.n) * d.jgroups * d.ublock0[p.nchild] : 0;
  d.units[2] = o.dv ? static_cast<int64_t>(p.n) * d.jgroups * p.nchild * d.vblocks : 0;
  const int64_t total = d.units[0] + d.units[1] + d.units[2];
  // (a launch holds fewer than 2^32 threads along x)
  constexpr int64_t kAcross = int64_t{1} << 20;
  const dim3 blocks(static_cast<uint32_t>(std::min(total, kAcross)), static_cast<uint32_t>((total + kAcross - 1) / kAcross));
  switch (JF) {
    case 1: gradient_kernel<1><<<blocks, 256, 0, stream>>>(d); break;
    case 2: gradient_kernel<2><<<blocks, 256, 0, stream>>>(d); break;
    case 4: gradient_kernel<4><<<blocks, 256, 0, stream>>>(d); break;
    default: gradient_kernel<8><<<blocks, 256, 0, stream>>>(d); break;
  }
  return hipGetLastError();
}

}  // namespace wl
