// Device pieces that the adapters' forward and backward passes share: tiles of
// tokens with one slot, their grouping, and accesses to rows of any width.
#pragma once

#include <algorithm>

#include "beside.h"
#include "coded.h"
#include "common.h"
#include "lds_dma.h"
#include "streams.h"

namespace wl {

namespace {

constexpr int kCUs = 256;
constexpr int kLeaderT = 256;    // most tokens without a grouping launch for workgroups of as many threads
constexpr int kMaxSlots = 4096;
constexpr int kGroupWaves = 8;   // slots of a grouping workgroup
constexpr int kStage = 8192;     // tokens whose slots it holds at a time

struct TileSource {
  const int32_t *index;  // [T]
  const int32_t *rank;   // [n] or null
  int32_t T, n, r;
  int32_t copies;        // tokens without an adapter are tiles too (y is not base)
  // grouped calls (else null): place i < max_tiles holds a tile's slot, count and
  // rank (count 0: no tile) and the tokens perm[i * M ..], -1 behind the last
  const int4 *tiles;
  const int32_t *perm;
  int32_t max_tiles;
};

struct Tile {
  int slot;   // -1: no adapter
  int count;  // tokens
  int rank;   // of the slot
  int rank16; // rounded up to 16
};

// A uniform value held in a scalar register.
__device__ __forceinline__ int keep(int v) { return __builtin_amdgcn_readfirstlane(v); }

// 16 bytes at a uniform address plus a lane's bytes: no arithmetic of the lanes.
__device__ __forceinline__ u32x4 ld16_at(const uint16_t *base, uint32_t bytes) {
  return *reinterpret_cast<const u32x4 *>(reinterpret_cast<const uint8_t *>(base) + bytes);
}

__device__ __forceinline__ u32x4 ld16_once_at(const uint16_t *base, uint32_t bytes) {
  return ld16_once(reinterpret_cast<const uint16_t *>(reinterpret_cast<const uint8_t *>(base) + bytes));
}

// Rank of a slot, in [0, r].
__device__ __forceinline__ int slot_rank(const int32_t *rank, int r, int a) {
  return rank ? min(max(rank[a], 0), r) : r;
}

// 16 bytes at an address that is 2-byte aligned (rows of an odd width): the
// memory path takes them whole.
typedef u32x4 u32x4_any __attribute__((aligned(2)));
__device__ __forceinline__ u32x4 ld16_any(const uint16_t *p) { return *reinterpret_cast<const u32x4_any *>(p); }
__device__ __forceinline__ u32x4 ld16_any_once(const uint16_t *p) {
  return __builtin_nontemporal_load(reinterpret_cast<const u32x4_any *>(p));
}
__device__ __forceinline__ void st16_any(uint16_t *p, u32x4 v) { *reinterpret_cast<u32x4_any *>(p) = v; }

// The first n of 8 bf16, zeros behind them.
__device__ __forceinline__ u32x4 first_of_8(u32x4 v, int n) {
  if (n >= 8) return v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] &= n >= 2 * i + 2 ? 0xffffffffu : n > 2 * i ? 0xffffu : 0u;
  return v;
}

// Up to 8 bf16 at p, of which `left` exist.
__device__ __forceinline__ u32x4 load_some(const uint16_t *p, int left) {
  u32x4 v{0u, 0u, 0u, 0u};
  if (left >= 8) return ld16_any(p);
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < left) v[e / 2] |= static_cast<uint32_t>(p[e]) << (16 * (e & 1));
  return v;
}

// The first `left` of 8 bf16 to p.
__device__ __forceinline__ void store_some(uint16_t *p, u32x4 v, int left) {
  if (left >= 8) return st16_any(p, v);
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < left) p[e] = static_cast<uint16_t>(v[e / 2] >> (16 * (e & 1)));
}

// 8 bf16 plus 8 floats, rounded once.
__device__ __forceinline__ u32x4 add_8(u32x4 v, f32x4 p, f32x4 q) {
  auto lo = [](uint32_t w) { return __uint_as_float(w << 16); };
  auto hi = [](uint32_t w) { return __uint_as_float(w & 0xffff0000u); };
  return u32x4{pack_bf16(lo(v[0]) + p[0], hi(v[0]) + p[1]), pack_bf16(lo(v[1]) + p[2], hi(v[1]) + p[3]),
               pack_bf16(lo(v[2]) + q[0], hi(v[2]) + q[1]), pack_bf16(lo(v[3]) + q[2], hi(v[3]) + q[3])};
}

// Place of tile t of n: hardware sends workgroup w to XCD w % 8 (the places are a
// multiple of 8), and each XCD has its own L2, so it gets neighbouring tiles, which
// share a slot: its V^T and U then come from one or two XCDs' L2 and not from all.
__device__ __forceinline__ int tile_place(int t, int n) {
  const int per = n >> 3, rem = n & 7, big = rem * (per + 1);
  const int x = t < big ? t / (per + 1) : rem + (t - big) / max(per, 1);
  return 8 * (t - (x * per + min(x, rem))) + x;
}
inline int tile_places(int64_t n) { return static_cast<int>((n + 7) & ~int64_t{7}); }

// Tile `id` of M tokens for a workgroup of 256 threads or more (of MOST, where there are
// so many tokens that are not grouped); its tokens go to tok (-1 behind the last).
// False (for the whole workgroup): nothing to do.
template <int M, int MOST = kLeaderT>
__device__ __forceinline__ bool get_tile(const TileSource &s, int id, Tile &t, int *tok) {
  if (s.tiles) {
    if (id >= s.max_tiles) return false;
    // one round of loads; the tokens of a tile that is not there are not used
    const int token = s.perm[static_cast<int64_t>(id) * M + threadIdx.x % M];
    const int4 e = s.tiles[id];
    if (e.y == 0) return false;
    t.slot = keep(e.x);
    t.count = keep(e.y);
    t.rank = keep(e.z);
    if (threadIdx.x < M) tok[threadIdx.x] = token;
  } else {
    if (id >= s.T) return false;
    __shared__ uint64_t member[MOST / 64];
    const int i = threadIdx.x, lane = i & 63, wave = i >> 6;
    // slots outside the pool count as slot n, no adapter
    const int of_id = s.index[id], of_i = i < s.T ? s.index[i] : 0;
    const int a = static_cast<uint32_t>(of_id) < static_cast<uint32_t>(s.n) ? of_id : s.n;
    const int b = static_cast<uint32_t>(of_i) < static_cast<uint32_t>(s.n) ? of_i : s.n;
    const uint64_t m = __builtin_amdgcn_ballot_w64(i < s.T && a == b);
    if (lane == 0 && wave < MOST / 64) member[wave] = m;
    if (i < M) tok[i] = -1;
    __syncthreads();
    int before = 0, at = 0, total = 0;  // members before token id, before token i, in all
#pragma unroll
    for (int w = 0; w < MOST / 64; ++w) {
      const uint64_t v = member[w];
      const int c = __builtin_popcountll(v);
      total += c;
      at += w < wave ? c : w == wave ? __builtin_popcountll(v & ((uint64_t{1} << lane) - 1)) : 0;
      before += w < (id >> 6) ? c : w == (id >> 6) ? __builtin_popcountll(v & ((uint64_t{1} << (id & 63)) - 1)) : 0;
    }
    if (before % M) return false;
    if (i < s.T && a == b && at >= before && at < before + M) tok[at - before] = i;
    t.slot = keep(a < s.n ? a : -1);
    t.count = keep(min(M, total - before));
    t.rank = t.slot >= 0 ? keep(slot_rank(s.rank, s.r, t.slot)) : 0;
    if (t.rank == 0) t.slot = -1;
  }
  t.rank16 = (t.rank + 15) & ~15;
  if (t.slot < 0 && !s.copies) return false;
  __syncthreads();
  return true;
}

// All tokens of a slot, in order, to list [kLeaderT], for a workgroup of 256 threads
// in a call that is not grouped; how many there are (0 for a slot of rank 0).
__device__ __forceinline__ int list_tokens(const TileSource &s, int slot, int *list) {
  __shared__ uint64_t of_slot[kLeaderT / 64];
  const int i = threadIdx.x, lane = i & 63, wave = i >> 6;
  const bool is = i < s.T && s.index[i < s.T ? i : 0] == slot;
  const uint64_t m = __builtin_amdgcn_ballot_w64(is);
  if (lane == 0) of_slot[wave] = m;
  const int rank = slot_rank(s.rank, s.r, slot);
  __syncthreads();
  int at = __builtin_popcountll(m & ((uint64_t{1} << lane) - 1)), total = 0;
#pragma unroll
  for (int w = 0; w < kLeaderT / 64; ++w) {
    const int c = __builtin_popcountll(of_slot[w]);
    at += w < wave ? c : 0;
    total += c;
  }
  if (is) list[at] = i;
  __syncthreads();
  return rank > 0 ? total : 0;
}

// Grouping of a long call.  A wave takes one slot (n: no adapter), or a workgroup
// does: it counts the tokens of every slot (the workgroup's histogram), so its first
// tile is known without waiting for anyone, and writes its tokens in ascending order.
// The slots of up to kStage tokens at a time sit in LDS, where all waves look
// through them, or each through its part.
struct GroupArgs {
  TileSource s;
  int4 *tiles;
  int32_t *perm;
  int32_t *first, *count;  // per slot [n]: its first tile and tokens (null: not wanted)
  int32_t *total;          // with these: how many tiles there are, items, and places
  // with these too: sums over a slot's tokens, in cuts of at most `cut` steps of 32 tokens:
  // slot, cut, how many cuts, and (more than one) the cut's place among all such cuts
  int4 *items;
  int4 *joins;             // of a place: slot, how many cuts (0 but at the slot's first)
  int32_t cut;
};

// Slots of up to kStage tokens from t0 on into LDS; eight loads at a time, none
// of them conditional, so that they leave back to back.  count(lane's slot) for
// each.
template <typename F>
__device__ __forceinline__ void stage_slots(const TileSource &s, int t0, int len, uint16_t *of, F &&count) {
  constexpr int W = kGroupWaves * 64, J = 8;
  for (int i0 = 0; i0 < len; i0 += J * W) {
    int32_t v[J];
#pragma unroll
    for (int j = 0; j < J; ++j) v[j] = s.index[t0 + min(i0 + j * W + static_cast<int>(threadIdx.x), len - 1)];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int i = i0 + j * W + static_cast<int>(threadIdx.x);
      if (i >= len) continue;
      const int a = static_cast<uint32_t>(v[j]) < static_cast<uint32_t>(s.n) ? v[j] : s.n;
      of[i] = static_cast<uint16_t>(a);
      count(a);
    }
  }
}

template <int M, bool SHARE>
__global__ __launch_bounds__(kGroupWaves * 64) void group_kernel(GroupArgs g) {
  const TileSource &s = g.s;
  __shared__ int hist[kMaxSlots + 1];
  __shared__ uint16_t of[kStage];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int mine = SHARE ? blockIdx.x : blockIdx.x * kGroupWaves + wave;
  const int id = SHARE ? threadIdx.x : lane, width = SHARE ? kGroupWaves * 64 : 64;  // of a slot's threads
  for (int b = threadIdx.x; b <= s.n; b += kGroupWaves * 64) hist[b] = 0;
  __syncthreads();
  for (int t0 = 0; t0 < s.T; t0 += kStage) {
    const int len = min(kStage, s.T - t0);
    stage_slots(s, t0, len, of, [&](int v) {
      // tokens of a sequence stand side by side: one addition for the lanes that
      // hold the first one's slot
      const int f = __builtin_amdgcn_readfirstlane(v);
      const uint64_t same = __builtin_amdgcn_ballot_w64(v == f);
      if (v != f)
        atomicAdd(&hist[v], 1);
      else if ((same & ((uint64_t{1} << lane) - 1)) == 0)
        atomicAdd(&hist[f], __builtin_popcountll(same));
    });
  }
  __syncthreads();
  __shared__ int tiles_of[kMaxSlots + 1];
  __shared__ uint16_t cuts_of[kMaxSlots + 1];  // (of steps of 32 tokens, 2^20 at most)
  for (int b = threadIdx.x; b <= s.n; b += kGroupWaves * 64) {
    const bool copy = b == s.n || slot_rank(s.rank, s.r, b) == 0;
    tiles_of[b] = copy && !s.copies ? 0 : (hist[b] + M - 1) / M;
    if (g.first) {
      const int steps = copy ? 0 : (hist[b] + 31) / 32;
      cuts_of[b] = static_cast<uint16_t>(b == s.n ? 0 : steps > g.cut ? (steps + g.cut - 1) / g.cut : 1);
    }
  }
  __syncthreads();
  const int cnt = mine <= s.n ? hist[mine] : 0, tiles = mine <= s.n ? tiles_of[mine] : 0;
  int tile0 = 0, total = 0, item0 = 0, place0 = 0;
  for (int b = lane; b <= s.n; b += 64) {
    const int k = tiles_of[b];
    total += k;
    tile0 += b < mine ? k : 0;
    const int c = g.first && b < mine ? cuts_of[b] : 0;
    item0 += c;
    place0 += c > 1 ? c : 0;
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    tile0 += __shfl_xor(tile0, d, 64);
    total += __shfl_xor(total, d, 64);
    item0 += __shfl_xor(item0, d, 64);
    place0 += __shfl_xor(place0, d, 64);
  }
  if (mine <= s.n) {
    const int rank = mine < s.n ? slot_rank(s.rank, s.r, mine) : 0, slot = rank > 0 ? mine : -1;
    for (int i = id; i < tiles; i += width) g.tiles[tile_place(tile0 + i, total)] = int4{slot, min(M, cnt - i * M), rank, 0};
    if (mine == s.n)
      for (int i = total + id; i < s.max_tiles; i += width) g.tiles[i] = int4{-1, 0, 0, 0};
    if (g.first && mine < s.n && id == 0) {
      g.first[mine] = tile0;
      g.count[mine] = slot >= 0 ? cnt : 0;
    }
    if (g.first && mine == s.n && id == 0) {
      g.total[0] = total;
      g.total[1] = item0;
      g.total[2] = place0;
    }
    if (g.first && mine < s.n) {
      const int cuts = cuts_of[mine];
      for (int q = id; q < cuts; q += width) {
        g.items[item0 + q] = int4{mine, q, cuts, place0 + q};
        if (cuts > 1) g.joins[place0 + q] = int4{mine, q == 0 ? cuts : 0, 0, 0};
      }
    }
    if (tiles) {
      int32_t *last = g.perm + static_cast<int64_t>(tile_place(tile0 + tiles - 1, total)) * M;
      for (int i = cnt - (tiles - 1) * M + id; i < M; i += width) last[i] = -1;
    }
  }
  // the tokens; every wave goes through every stage (the barriers are the workgroup's)
  __shared__ int part[kGroupWaves];
  int before = 0;  // the slot's tokens in the stages so far
  for (int t0 = 0; t0 < s.T; t0 += kStage) {
    const int len = min(kStage, s.T - t0);
    if (s.T > kStage) {
      __syncthreads();
      stage_slots(s, t0, len, of, [](int) {});
      __syncthreads();
    }
    if (!tiles) continue;
    auto look = [&](int i0, int end, uint64_t (&hits)[8]) {
      uint64_t any = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = i0 + 64 * j + lane;
        const int v = of[min(i, end - 1)];
        hits[j] = __builtin_amdgcn_ballot_w64(i < end && v == mine);
        any |= hits[j];
      }
      return any;
    };
    int found = before, from = 0, end = len;
    if constexpr (SHARE) {  // a wave's part of the stage, and what the parts before it hold
      const int per = (len + kGroupWaves - 1) / kGroupWaves;
      from = min(wave * per, len);
      end = min(from + per, len);
      int c = 0;
      for (int i0 = from; i0 < end; i0 += 512) {
        uint64_t hits[8];
        look(i0, end, hits);
#pragma unroll
        for (int j = 0; j < 8; ++j) c += __builtin_popcountll(hits[j]);
      }
      if (lane == 0) part[wave] = c;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kGroupWaves; ++w) {
        found += w < wave ? part[w] : 0;
        before += part[w];
      }
    }
    for (int i0 = from; i0 < end && found < cnt; i0 += 512) {
      uint64_t hits[8];
      if (!look(i0, end, hits)) continue;  // (the most common case: sequences are long, and slots many)
      // places of the tiles that these 512 tokens can fall in, a lane each
      const int tile = found / M, place = tile_place(min(tile0 + tile + lane, total - 1), total);
      static_assert(512 / M + 1 <= 64, "a lane for each tile");
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint64_t m = hits[j], below = (uint64_t{1} << lane) - 1;
        const int at = found + __builtin_popcountll(m & below);
        const int to = __shfl(place, at / M - tile, 64) * M + at % M;
        if (m >> lane & 1) g.perm[to] = t0 + i0 + 64 * j + lane;
        found += __builtin_popcountll(m);
      }
    }
    if constexpr (!SHARE) before = found;
  }
}

// A workgroup for each slot while they all run at once (two on a CU) and there is
// something to share (4096 tokens 8.9 -> 6.9 us, 77 tokens 4.4 -> 5.2); else a wave.
constexpr int kShareSlots = 2 * kCUs, kShareTokens = 512;
template <int M>
hipError_t launch_group(const GroupArgs &g, hipStream_t stream) {
  if (g.s.n < kShareSlots && g.s.T > kShareTokens)
    group_kernel<M, true><<<g.s.n + 1, kGroupWaves * 64, 0, stream>>>(g);
  else
    group_kernel<M, false><<<(g.s.n + kGroupWaves) / kGroupWaves, kGroupWaves * 64, 0, stream>>>(g);
  return hipGetLastError();
}

// z and g enter the second products as kParts bf16 each: what the first leaves of the
// float goes to the next, and three of 8 significant bits hold all 24 (each is cut off, not
// rounded, so nothing is left over; an infinity or NaN is the first part alone).
constexpr int kParts = 3;
__device__ __forceinline__ void split4(f32x4 v, u32x2 (&o)[kParts]) {
#pragma unroll
  for (int p = 0; p < kParts; ++p) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = __float_as_uint(v[i]) & 0xffff0000u;
      const float d = v[i] - __uint_as_float(w[i]);
      v[i] = fabsf(d) < __builtin_inff() ? d : 0.f;
    }
    o[p] = u32x2{w[0] >> 16 | w[1], w[2] >> 16 | w[3]};
  }
}

// The parts of four floats to `to`, `next` elements apart.
__device__ __forceinline__ void store_parts(f32x4 v, uint16_t *to, int next) {
  u32x2 o[kParts];
  split4(v, o);
#pragma unroll
  for (int p = 0; p < kParts; ++p) *reinterpret_cast<u32x2 *>(to + p * next) = o[p];
}

inline size_t align256(size_t n) { return (n + 255) & ~size_t{255}; }

}  // namespace

}  // namespace wl
