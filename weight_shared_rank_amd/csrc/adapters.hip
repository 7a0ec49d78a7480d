// Low-rank adapters of many requests at once beside one shared projection.
//
//   z_t = V_a^T x_t,   y_t = base_t + c_a U_a z_t,   a = index[t]
//
// with U_a [N][r], V_a^T [r][K] of slot a in the pool; a stacked call's children
// have their own U and V over one x.  Tokens without an adapter keep base.
//
// Tokens are taken in tiles of up to M that share a slot, so that an adapter is
// read once for M tokens and its products run on the matrix cores: the tokens
// are the columns of a product, the rows of V^T or U its rows.  Where a call has
// few tokens (kLeaderT) there is nothing to prepare: workgroup t looks through
// the whole index and works if token t is the first, the 17th, ... of its slot.
// A longer call is grouped first (group_kernel).
//
// Two launches: thin_kernel gives z in float32 (K cut into slices that the
// reader adds up in a fixed order), expand_kernel turns c z into a pair of bf16
// (the value and what its rounding left, 16 significant bits), multiplies by U
// and adds base, rounding once.
//
// What bounds it: few tokens, reading the adapters in use; many, reading and
// writing base and y.  The products are far below the matrix cores' rate.
#include <algorithm>
#include <type_traits>

#include "beside.h"
#include "coded.h"
#include "common.h"
#include "lds_dma.h"

namespace wl {

namespace {

constexpr int kCUs = 256;
constexpr int kLeaderT = 256;    // up to here no grouping launch (a thread of a workgroup for each token)
constexpr int kLeaderM = 16;     // tokens of a tile there
constexpr int kMaxSlots = 4096;
constexpr int kStage = 8192;     // tokens whose slots a grouping workgroup holds at a time

struct TileSource {
  const int32_t *index;  // [T]
  const int32_t *rank;   // [n] or null
  int32_t T, n, r;
  int32_t copies;        // tokens without an adapter are tiles too (y is not base)
  // grouped calls (else null): tile i has the slot and count tiles[i] and the
  // tokens perm[i * M ..], -1 behind the last
  const int2 *tiles;
  const int32_t *ntiles;
  const int32_t *perm;
};

struct Tile {
  int slot;   // -1: no adapter
  int count;  // tokens
  int rank;   // of the slot
  int rank16; // rounded up to 16
};

// Rank of a slot, in [0, r].
__device__ __forceinline__ int slot_rank(const int32_t *rank, int r, int a) {
  return rank ? min(max(rank[a], 0), r) : r;
}

// The first n of 8 bf16, zeros behind them.
__device__ __forceinline__ u32x4 first_of_8(u32x4 v, int n) {
  if (n >= 8) return v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] &= n >= 2 * i + 2 ? 0xffffffffu : n > 2 * i ? 0xffffu : 0u;
  return v;
}

// Tile `id` of M tokens for a workgroup of 256 threads; its tokens go to tok
// (-1 behind the last).  False (for the whole workgroup): nothing to do.
template <int M>
__device__ __forceinline__ bool get_tile(const TileSource &s, int id, Tile &t, int *tok) {
  if (s.tiles) {
    if (id >= *s.ntiles) return false;
    const int2 e = s.tiles[id];
    t.slot = e.x;
    t.count = e.y;
    if (threadIdx.x < M) tok[threadIdx.x] = s.perm[static_cast<int64_t>(id) * M + threadIdx.x];
  } else {
    __shared__ uint64_t member[kLeaderT / 64];
    const int i = threadIdx.x, lane = i & 63, wave = i >> 6;
    // slots outside the pool count as slot n, no adapter
    const int of_id = s.index[id], of_i = i < s.T ? s.index[i] : 0;
    const int a = static_cast<uint32_t>(of_id) < static_cast<uint32_t>(s.n) ? of_id : s.n;
    const int b = static_cast<uint32_t>(of_i) < static_cast<uint32_t>(s.n) ? of_i : s.n;
    const uint64_t m = __builtin_amdgcn_ballot_w64(i < s.T && a == b);
    if (lane == 0) member[wave] = m;
    if (i < M) tok[i] = -1;
    __syncthreads();
    int before = 0, at = 0, total = 0;  // members before token id, before token i, in all
#pragma unroll
    for (int w = 0; w < kLeaderT / 64; ++w) {
      const uint64_t v = member[w];
      const int c = __builtin_popcountll(v);
      total += c;
      at += w < wave ? c : w == wave ? __builtin_popcountll(v & ((uint64_t{1} << lane) - 1)) : 0;
      before += w < (id >> 6) ? c : w == (id >> 6) ? __builtin_popcountll(v & ((uint64_t{1} << (id & 63)) - 1)) : 0;
    }
    if (before % M) return false;
    if (i < s.T && a == b && at >= before && at < before + M) tok[at - before] = i;
    t.slot = a < s.n ? a : -1;
    t.count = min(M, total - before);
  }
  t.rank = 0;
  if (t.slot >= 0) {
    t.rank = slot_rank(s.rank, s.r, t.slot);
    if (t.rank == 0) t.slot = -1;
  }
  t.rank16 = (t.rank + 15) & ~15;
  if (t.slot < 0 && !s.copies) return false;
  __syncthreads();
  return true;
}

// Grouping of a long call.  A wave takes one slot (n: no adapter): it counts the
// tokens of every slot (the workgroup's histogram), so its first tile is known
// without waiting for anyone, and writes its tokens in ascending order.  The
// slots of up to kStage tokens at a time sit in LDS, where all four waves look
// through them.
struct GroupArgs {
  TileSource s;
  int2 *tiles;
  int32_t *ntiles, *perm;
  int32_t *first, *count;  // per slot [n]: its first tile and tokens (null: not wanted)
};

__device__ __forceinline__ uint16_t stage_slot(const TileSource &s, int64_t t) {
  const uint32_t v = static_cast<uint32_t>(s.index[t]);
  return static_cast<uint16_t>(v < static_cast<uint32_t>(s.n) ? v : s.n);
}

template <int M>
__global__ __launch_bounds__(256) void group_kernel(GroupArgs g) {
  const TileSource &s = g.s;
  __shared__ int hist[kMaxSlots + 1];
  __shared__ uint16_t of[kStage];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int mine = blockIdx.x * 4 + wave;
  for (int b = threadIdx.x; b <= s.n; b += 256) hist[b] = 0;
  __syncthreads();
  for (int t0 = 0; t0 < s.T; t0 += kStage) {
    const int len = min(kStage, s.T - t0);
#pragma unroll 8
    for (int i = threadIdx.x; i < len; i += 256) {
      const uint16_t v = stage_slot(s, t0 + i);
      of[i] = v;
      atomicAdd(&hist[v], 1);
    }
  }
  __syncthreads();
  const int cnt = mine <= s.n ? hist[mine] : 0;
  int tile0 = 0, tiles = 0;
  for (int b = lane; b <= min(mine, s.n); b += 64) {
    const bool copy = b == s.n || slot_rank(s.rank, s.r, b) == 0;
    const int k = copy && !s.copies ? 0 : (hist[b] + M - 1) / M;
    if (b < mine)
      tile0 += k;
    else
      tiles = k;
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    tile0 += __shfl_xor(tile0, d, 64);
    tiles += __shfl_xor(tiles, d, 64);
  }
  if (mine <= s.n) {
    const int slot = mine < s.n && slot_rank(s.rank, s.r, mine) > 0 ? mine : -1;
    for (int i = lane; i < tiles; i += 64) g.tiles[tile0 + i] = int2{slot, min(M, cnt - i * M)};
    if (mine == s.n && lane == 0) *g.ntiles = tile0 + tiles;
    if (g.first && mine < s.n && lane == 0) {
      g.first[mine] = tile0;
      g.count[mine] = slot >= 0 ? cnt : 0;
    }
    for (int i = cnt + lane; i < tiles * M; i += 64) g.perm[static_cast<int64_t>(tile0) * M + i] = -1;
  }
  // the tokens; every wave goes through every stage (the barriers are the workgroup's)
  int found = 0;
  int32_t *out = g.perm + static_cast<int64_t>(tile0) * M;
  for (int t0 = 0; t0 < s.T; t0 += kStage) {
    const int len = min(kStage, s.T - t0);
    if (s.T > kStage) {
      __syncthreads();
      for (int i = threadIdx.x; i < len; i += 256) of[i] = stage_slot(s, t0 + i);
      __syncthreads();
    }
    if (!tiles) continue;
    for (int i0 = 0; i0 < len && found < cnt; i0 += 256) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = i0 + 64 * j + lane;
        const bool hit = i < len && of[i] == mine;
        const uint64_t m = __builtin_amdgcn_ballot_w64(hit);
        if (hit) out[found + __builtin_popcountll(m & ((uint64_t{1} << lane) - 1))] = t0 + i;
        found += __builtin_popcountll(m);
      }
    }
  }
}

// ---- thin products ------------------------------------------------------------
// P[slice][row][col] = sum over the slice's k of A_a[col][k] x[token][k]: A the
// rows of V^T of all children.  A workgroup takes a tile of 16 MF tokens, a
// K slice and up to 16 NF rows of A; its four waves take steps of 64 k in turn
// and meet in LDS.  16-row tiles past a slot's rank are left out.  Both operands go
// straight to registers: a lane's two loads of a step are 32 neighbouring bytes
// of its row, four lanes a cache line.
struct ThinArgs {
  TileSource s;
  const uint16_t *x;   // [T][K]
  const uint16_t *A;   // [n][nchild * r][K]
  int32_t K, nchild;
  int32_t slices, per; // slices of K, steps of each
  float *P;            // [slices][rows][R]
  int32_t R;           // nchild * r
  int64_t rows;
};

template <int MF, int NF>
__global__ __launch_bounds__(256) void thin_kernel(ThinArgs a) {
  constexpr int M = 16 * MF;
  __shared__ int tok[M];
  __shared__ f32x4 part[3][MF * NF][64];
  Tile t;
  if (!get_tile<M>(a.s, blockIdx.x, t, tok) || t.slot < 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r16 = lane & 15, g = lane >> 4;
  const int per_child = t.rank16 / 16, live = a.nchild * per_child;  // 16-row tiles of A in use
  const int f0 = blockIdx.z * NF;
  if (f0 >= live) return;
  const uint16_t *xr[MF], *ar[NF];
  bool xin[MF];
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    const int token = tok[16 * i + r16];
    xin[i] = token >= 0;
    xr[i] = a.x + static_cast<int64_t>(max(token, 0)) * a.K;
  }
  int col[NF];  // first row of A (column of P) of a tile
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    const int v = min(f0 + f, live - 1);  // tiles past the last repeat it and are not stored
    col[f] = (v / per_child) * a.s.r + (v % per_child) * 16;
    ar[f] = a.A + (static_cast<int64_t>(t.slot) * a.R + col[f] + r16) * a.K;
  }
  f32x4 acc[NF][MF];
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int i = 0; i < MF; ++i) acc[f][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  const u32x4 zero{0u, 0u, 0u, 0u};
  const int steps = (a.K + 63) / 64;
  const int end = min(steps, static_cast<int>(blockIdx.y + 1) * a.per);
  u32x4 xv[2][MF][2], av[2][NF][2];
  auto load = [&](int step, u32x4(&xo)[MF][2], u32x4(&ao)[NF][2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = step * 64 + g * 16 + h * 8;
      const bool in = step < end && k < a.K;
#pragma unroll
      for (int f = 0; f < NF; ++f) ao[f][h] = in ? ld16(ar[f] + k) : zero;
#pragma unroll
      for (int i = 0; i < MF; ++i) xo[i][h] = in && xin[i] ? ld16(xr[i] + k) : zero;
    }
  };
  auto multiply = [&](const u32x4(&xo)[MF][2], const u32x4(&ao)[NF][2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int i = 0; i < MF; ++i) acc[f][i] = mfma16x16x32(ao[f][h], xo[i][h], acc[f][i]);
  };
  int step = blockIdx.y * a.per + wave;
  load(step, xv[0], av[0]);
  for (; step < end; step += 8) {
    load(step + 4, xv[1], av[1]);
    multiply(xv[0], av[0]);
    load(step + 8, xv[0], av[0]);
    multiply(xv[1], av[1]);
  }
  if (wave > 0) {
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int i = 0; i < MF; ++i) part[wave - 1][f * MF + i][lane] = acc[f][i];
  }
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      f32x4 v = acc[f][i];
#pragma unroll
      for (int w = 0; w < 3; ++w) v += part[w][f * MF + i][lane];
      const int c = 16 * i + r16;
      if (f0 + f >= live || c >= t.count) continue;
      const int64_t row = a.s.tiles ? static_cast<int64_t>(blockIdx.x) * M + c : tok[c];
      *reinterpret_cast<f32x4 *>(a.P + (blockIdx.y * a.rows + row) * a.R + col[f] + g * 4) = v;
    }
}

// ---- the products with U, and base ---------------------------------------------
// y[t][n] = base[t][n] + sum_j c z[t][j] U_a[n][j].  A wave takes 64 n at a time,
// `turns` times, as four row tiles whose rows are numbered so that a lane ends
// up with 8 neighbouring n of its token twice: base and y move as 16 bytes a
// lane, 64 to a row and load.  c z is the workgroup's, as a pair of bf16 in LDS.
struct ExpandArgs {
  TileSource s;
  const float *P;        // [slices][rows][R]
  int32_t slices, R;
  int64_t rows;
  const float *scale;    // [n]
  const uint16_t *U;     // [n][Ntot][r]
  const uint16_t *base;  // [T][Ntot]
  uint16_t *y;           // [T][Ntot]
  int32_t Ntot, nchild, turns;
  int32_t N[kMaxChildren], n0[kMaxChildren];  // rows and first row of a child
  int32_t block0[kMaxChildren];               // first workgroup (x) of a child
  int32_t aligned[kMaxChildren];              // its columns of base and y are 16-byte aligned
};

// What a float leaves over its bf16: 0 for infinity and NaN.
__device__ __forceinline__ float left_over(float v, uint16_t h) {
  const float d = v - bf16_to_f32(h);
  return fabsf(d) < __builtin_inff() ? d : 0.f;
}

template <int MF>
__global__ __launch_bounds__(256) void expand_kernel(ExpandArgs a) {
  constexpr int M = 16 * MF;
  __shared__ int tok[M];
  extern __shared__ __align__(16) uint16_t zs[];  // [2][M][pitch]
  Tile t;
  if (!get_tile<M>(a.s, blockIdx.y, t, tok)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r16 = lane & 15, g = lane >> 4;
  int c = 0;
#pragma unroll
  for (int i = 1; i < kMaxChildren; ++i)
    if (i < a.nchild && static_cast<int>(blockIdx.x) >= a.block0[i]) c = i;
  const int N = a.N[c], r = a.s.r;
  const int first = (static_cast<int>(blockIdx.x) - a.block0[c]) * a.turns * 256;
  const bool adapted = t.slot >= 0;
  const int pitch = r + 8;  // 16 bytes more than the row: fragment reads spread over the banks
  if (adapted) {
    const float scale = a.scale[t.slot];
    const int quads = t.rank16 / 4;
    for (int i = threadIdx.x; i < M * quads; i += 256) {
      const int m = i / quads, j = (i % quads) * 4;
      f32x4 v{0.f, 0.f, 0.f, 0.f};
      if (m < t.count) {
        const int64_t row = a.s.tiles ? static_cast<int64_t>(blockIdx.y) * M + m : tok[m];
        const float *p = a.P + row * a.R + c * r + j;
        for (int sl = 0; sl < a.slices; ++sl) v += *reinterpret_cast<const f32x4 *>(p + sl * a.rows * a.R);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = j + k < t.rank ? v[k] * scale : 0.f;
      uint16_t h[4], l[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        h[k] = f32_to_bf16(v[k]);
        l[k] = f32_to_bf16(left_over(v[k], h[k]));
      }
      *reinterpret_cast<u32x2 *>(zs + m * pitch + j) = u32x2{h[0] | static_cast<uint32_t>(h[1]) << 16, h[2] | static_cast<uint32_t>(h[3]) << 16};
      *reinterpret_cast<u32x2 *>(zs + (M + m) * pitch + j) = u32x2{l[0] | static_cast<uint32_t>(l[1]) << 16, l[2] | static_cast<uint32_t>(l[3]) << 16};
    }
    __syncthreads();
  }
  const u32x4 zero{0u, 0u, 0u, 0u};
  const int lrow = 8 * (r16 >> 2) + (r16 & 3);
  for (int turn = 0; turn < a.turns; ++turn) {
    const int nw = first + (turn * 4 + wave) * 64;
    if (nw >= N) break;
    // base: [token tile][half of the 64 n]
    u32x4 b[MF][2];
    bool whole[2];
    int64_t at[MF];
#pragma unroll
    for (int h = 0; h < 2; ++h) whole[h] = a.aligned[c] && nw + 32 * h + 8 * g + 8 <= N;
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      const int token = tok[16 * i + r16];
      at[i] = token < 0 ? -1 : static_cast<int64_t>(token) * a.Ntot + a.n0[c] + nw + 8 * g;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        b[i][h] = zero;
        if (token >= 0 && whole[h]) {
          b[i][h] = ld16(a.base + at[i] + 32 * h);
        } else if (token >= 0) {
          const int lim = N - (nw + 32 * h + 8 * g);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (e < lim) b[i][h][e / 2] |= static_cast<uint32_t>(a.base[at[i] + 32 * h + e]) << (16 * (e & 1));
        }
      }
    }
    if (adapted) {
      f32x4 acc[4][MF];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < MF; ++i) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};
      const uint16_t *U = a.U + (static_cast<int64_t>(t.slot) * a.Ntot + a.n0[c]) * r;
      for (int k = 8 * g; k - 8 * g < t.rank16; k += 32) {
        u32x4 uv[4], zv[MF][2];
        const bool in = k < t.rank16;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int n = nw + 32 * (j >> 1) + lrow + 4 * (j & 1);
          uv[j] = in && n < N ? ld16(U + static_cast<int64_t>(n) * r + k) : zero;
        }
        if (k + 8 > t.rank) {
#pragma unroll
          for (int j = 0; j < 4; ++j) uv[j] = first_of_8(uv[j], t.rank - k);
        }
#pragma unroll
        for (int i = 0; i < MF; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) zv[i][h] = in ? ld16(zs + (h * M + 16 * i + r16) * pitch + k) : zero;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < MF; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[j][i] = mfma16x16x32(uv[j], zv[i][h], acc[j][i]);
      }
#pragma unroll
      for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const f32x4 p = acc[2 * h][i], q = acc[2 * h + 1][i];
          u32x4 &v = b[i][h];
          v = u32x4{pack_bf16(__uint_as_float(v[0] << 16) + p[0], __uint_as_float(v[0] & 0xffff0000u) + p[1]),
                    pack_bf16(__uint_as_float(v[1] << 16) + p[2], __uint_as_float(v[1] & 0xffff0000u) + p[3]),
                    pack_bf16(__uint_as_float(v[2] << 16) + q[0], __uint_as_float(v[2] & 0xffff0000u) + q[1]),
                    pack_bf16(__uint_as_float(v[3] << 16) + q[2], __uint_as_float(v[3] & 0xffff0000u) + q[3])};
        }
    }
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (at[i] < 0) continue;
        if (whole[h]) {
          *reinterpret_cast<u32x4 *>(a.y + at[i] + 32 * h) = b[i][h];
        } else {
          const int lim = N - (nw + 32 * h + 8 * g);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (e < lim) a.y[at[i] + 32 * h + e] = static_cast<uint16_t>(b[i][h][e / 2] >> (16 * (e & 1)));
        }
      }
  }
}

// ---- plan ----------------------------------------------------------------------

constexpr int kGroupMF = 2;  // token fragments of a tile of a grouped call

struct Plan {
  bool grouped;
  int M, tiles;          // tokens of a tile, most tiles there can be
  int NF, zgroups;       // thin: 16-row tiles of a workgroup, workgroups for all rows
  int slices, per;
  int64_t rows;          // rows of P
  size_t tiles_at, perm_at, p_at, bytes;
};

size_t align256(size_t n) { return (n + 255) & ~size_t{255}; }

Plan make_plan(const AdapterPool &p, int T) {
  Plan q{};
  q.grouped = T > kLeaderT;
  q.M = q.grouped ? 16 * kGroupMF : kLeaderM;
  q.tiles = q.grouped ? T / q.M + std::min(p.n + 1, T) : T;
  const int row_tiles = p.nchild * p.r / 16;
  q.NF = row_tiles >= 8 ? 8 : row_tiles >= 3 ? 4 : row_tiles;
  q.zgroups = (row_tiles + q.NF - 1) / q.NF;
  // K slices until the workgroups fill the CUs a few times over, none shorter
  // than a step for each wave
  const int steps = (p.K + 63) / 64;
  const int busy = (q.grouped ? (T + q.M - 1) / q.M : T) * q.zgroups;
  int want = std::min({8, (4 * kCUs + busy - 1) / busy, (steps + 3) / 4});
  q.per = (steps + want - 1) / want;
  q.slices = (steps + q.per - 1) / q.per;
  q.rows = q.grouped ? static_cast<int64_t>(q.tiles) * q.M : T;
  q.tiles_at = 256;  // ntiles first
  q.perm_at = q.tiles_at + (q.grouped ? align256(sizeof(int2) * q.tiles) : 0);
  q.p_at = q.perm_at + (q.grouped ? align256(sizeof(int32_t) * q.rows) : 0);
  q.bytes = q.p_at + align256(sizeof(float) * q.slices * q.rows * p.nchild * p.r);
  return q;
}

template <int MF>
hipError_t launch_thin(const ThinArgs &a, const Plan &q, hipStream_t stream) {
  const dim3 grid(q.tiles, q.slices, q.zgroups);
  switch (q.NF) {
    case 1: thin_kernel<MF, 1><<<grid, 256, 0, stream>>>(a); break;
    case 2: thin_kernel<MF, 2><<<grid, 256, 0, stream>>>(a); break;
    case 4: thin_kernel<MF, 4><<<grid, 256, 0, stream>>>(a); break;
    default: thin_kernel<MF, 8><<<grid, 256, 0, stream>>>(a); break;
  }
  return hipGetLastError();
}

}  // namespace

size_t adapters_workspace_bytes(const AdapterPool &p, int T) { return T > 0 ? make_plan(p, T).bytes : 256; }

hipError_t launch_adapters(const AdapterPool &p, const uint16_t *x, const int32_t *index, int T, const uint16_t *base,
                           uint16_t *y, void *ws, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  const Plan q = make_plan(p, T);
  uint8_t *w = static_cast<uint8_t *>(ws);
  TileSource s{};
  s.index = index;
  s.rank = p.rank;
  s.T = T;
  s.n = p.n;
  s.r = p.r;
  s.copies = base != y;
  hipError_t e = hipSuccess;
  if (q.grouped) {
    GroupArgs g{};
    g.s = s;
    g.ntiles = reinterpret_cast<int32_t *>(w);
    g.tiles = reinterpret_cast<int2 *>(w + q.tiles_at);
    g.perm = reinterpret_cast<int32_t *>(w + q.perm_at);
    group_kernel<16 * kGroupMF><<<(p.n + 4) / 4, 256, 0, stream>>>(g);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    s.tiles = g.tiles;
    s.ntiles = g.ntiles;
    s.perm = g.perm;
  }
  ThinArgs t{};
  t.s = s;
  t.x = x;
  t.A = p.vt;
  t.K = p.K;
  t.nchild = p.nchild;
  t.slices = q.slices;
  t.per = q.per;
  t.P = reinterpret_cast<float *>(w + q.p_at);
  t.R = p.nchild * p.r;
  t.rows = q.rows;
  e = q.grouped ? launch_thin<kGroupMF>(t, q, stream) : launch_thin<1>(t, q, stream);
  if (e != hipSuccess) return e;
  ExpandArgs a{};
  a.s = s;
  a.P = t.P;
  a.slices = q.slices;
  a.R = t.R;
  a.rows = q.rows;
  a.scale = p.scale;
  a.U = p.u;
  a.base = base;
  a.y = y;
  a.Ntot = p.Ntot;
  a.nchild = p.nchild;
  int blocks = 0;
  for (int c = 0; c < p.nchild; ++c) blocks += (p.N[c] + 255) / 256;
  const int busy = q.grouped ? (T + q.M - 1) / q.M : T;
  a.turns = std::max(1, std::min<int>(8, static_cast<int>(static_cast<int64_t>(blocks) * busy / (8 * kCUs))));
  blocks = 0;
  const bool rows16 = p.Ntot % 8 == 0 && reinterpret_cast<uintptr_t>(base) % 16 == 0 && reinterpret_cast<uintptr_t>(y) % 16 == 0;
  for (int c = 0, n0 = 0; c < p.nchild; ++c) {
    a.N[c] = p.N[c];
    a.n0[c] = n0;
    a.block0[c] = blocks;
    a.aligned[c] = rows16 && n0 % 8 == 0;
    blocks += (p.N[c] + 256 * a.turns - 1) / (256 * a.turns);
    n0 += p.N[c];
  }
  const dim3 grid(blocks, q.tiles);
  const size_t lds = sizeof(uint16_t) * 2 * q.M * (p.r + 8);
  if (q.grouped)
    expand_kernel<kGroupMF><<<grid, 256, lds, stream>>>(a);
  else
    expand_kernel<1><<<grid, 256, lds, stream>>>(a);
  return hipGetLastError();
}

}  // namespace wl
