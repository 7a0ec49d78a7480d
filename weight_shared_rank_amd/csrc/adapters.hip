// Low-rank adapters of many requests at once beside one shared projection.
//
//   z_t = V_a^T x_t,   y_t = base_t + c_a U_a z_t,   a = index[t]
//
// with U_a [N][r], V_a^T [r][K] of slot a in the pool; a stacked call's children
// have their own U and V over one x.  Tokens without an adapter keep base.
//
// Tokens are taken in tiles that share a slot: the columns of matrix products whose
// rows are V^T's and U's.  c z enters the second product in three parts of bf16, which
// hold all of its float32; y is rounded once.
//
// Few tokens: nothing is prepared and there is one launch, few_kernel.  Workgroup t
// looks through the whole index and works if token t is the first, the 17th, ... of its
// slot.  It makes z of its tile itself, as do the others along the children's rows: V^T
// comes from L2 then, and a launch that hands z over costs more (64 tokens through
// gate|up of 2 x 21504 x 5376 at rank 16: 7.5 + 25 us in two).
// More tokens: a grouping (group_kernel) tells few_kernel the tiles.
// Many tokens, or a high rank: the grouping, z in float32 slices of K (thin_kernel), the
// products with U and base (expand_kernel), in tiles of 64 tokens; between them, where
// many workgroups would add up the same slices, finish_kernel.
//
// Measured: 1 token through 1B q|k|v 5.6 us, of which a launch is most; 64 tokens of 57
// adapters through 31B gate|up 27 (103 MB read, 114 moved); 4096 tokens of 12 through 31B
// o at rank 64 6.6 + 19 + 5 + 26.6 (thin_kernel 80 MB at 4.2 TB/s, expand_kernel 100 at 3.8).
//
// Everything moves as rows, 8 lanes to a cache line, and reaches the matrix cores
// through LDS: fragments loaded as they are used (16 rows of 64 bytes a load) pass
// the first-level cache at a quarter of the rate (9.5 against 35 TB/s over the
// card).  The loops are short, so what surrounds their loads counts: none is
// conditional and no path leaves a loop early (where paths meet, the compiler cannot
// count the loads in flight and waits for all of them), addresses are a scalar plus
// a fixed offset of the lane, and what masks a partial stage or row is kept apart.
//
// What bounds it: few tokens, reading the adapters in use; many, reading and
// writing base and y.  The products are far below the matrix cores' rate.
#include "adapter_factors.h"

namespace wl {

namespace {

constexpr int kTileM = 16;  // tokens of a tile of a call of few tokens

struct AdapterArgs {
  TileSource s;
  const uint16_t *x;     // [T][K]
  const uint16_t *vt;    // [n][nchild * r][K]
  const uint16_t *u;     // [n][Ntot][r]
  const float *scale;    // [n]
  const uint16_t *base;  // [T][Ntot]
  uint16_t *y;           // [T][Ntot]
  const float *P;        // grouped calls: z [slices][rows][R]
  int64_t rows;
  int32_t R, slices;     // R: nchild * r
  const uint16_t *z;     // or c z, the rows of Factors, of RC chunks of a child
  int32_t RC;
  int32_t K, Ntot, nchild, turns;             // turns: times a wave takes 64 rows of U
  int32_t N[kMaxChildren], n0[kMaxChildren];  // rows and first row of a child
  int32_t block0[kMaxChildren];               // first workgroup (y) of a child
};

// Elements of a row of c z in LDS: as many ranks as RowWalk reads at most (a power
// of two, 32 or more), and 16 bytes more, which spread the fragment reads over the
// banks.
__host__ __device__ constexpr int z_pitch(int r) { return (r <= 32 ? 32 : r <= 64 ? 64 : r <= 128 ? 128 : 256) + 8; }

// c z of NF row tiles of V^T (from row j0 of the slot's child on) to zs [kParts][16][pitch].
// A stage is KS values of k: rows of 64 k (128 bytes), chunk c of row t in slot
// c ^ t % 8, so that fragment reads touch every bank.  It waits in registers while
// the kDeep - 1 before it are used.  A wave multiplies two row tiles (one where there
// is no more) over 32 k of a stage: what it reads of LDS bounds the loop.  The waves'
// sums meet in LDS in wave order.
// (A stage of 20 KB with conditional loads: 0.42 us, with masks and 64-bit addresses
// throughout 0.39, as it is 0.27.)
template <int NF>
__device__ __forceinline__ void form_z(const AdapterArgs &a, const Tile &t, const int *tok, int c, int j0, uint8_t *lds,
                                       uint16_t *zs) {
  constexpr int FR = NF == 1 ? 1 : 2, FP = NF / FR, H = kWaves / FP;  // row tiles of a wave, pairs, waves along k
  constexpr int KS = 32 * H, SUBS = KS / 64;
  constexpr int XB = SUBS * kTileM * 128, AB = SUBS * NF * 2048, STAGE = XB + AB;  // bytes of a stage
  constexpr int AP = AB / 16 / kThreads;                                           // pieces of V^T of a thread
  static_assert(XB / 16 <= kThreads && AP * kThreads * 16 == AB && kDeep % 2 == 0, "stage shape");
  const int lane = threadIdx.x & 63, wave = keep(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4, K = a.K;
  const u32x4 zero{0u, 0u, 0u, 0u};
  // pieces of 16 bytes: 64 k (sub), row, chunk
  const int chunk = threadIdx.x & 7;
  const int xrow = threadIdx.x / 8 % kTileM, xsub = threadIdx.x / (8 * kTileM) % SUBS;  // (NF 4: every piece twice)
  const int xtoken = tok[xrow] < 0 ? tok[0] : tok[xrow];  // (columns without a token are not stored)
  const uint16_t *xrowp = a.x + static_cast<int64_t>(xtoken) * K;
  const int xk = xsub * 64 + chunk * 8;
  const uint16_t *av0 = a.vt + ((static_cast<int64_t>(t.slot) * a.nchild + c) * a.s.r + j0) * K;
  uint32_t arow[AP];  // bytes from av0 to the piece's row; row tiles past the slot's rank repeat the last (masked)
  int ak[AP];
  uint8_t *aput[AP];
#pragma unroll
  for (int i = 0; i < AP; ++i) {
    const int p = i * kThreads + static_cast<int>(threadIdx.x), row = p / 8 % (16 * NF), sub = p / (128 * NF);
    arow[i] = static_cast<uint32_t>(min(row, t.rank16 - 1 - j0)) * static_cast<uint32_t>(K) * 2u;
    ak[i] = sub * 64 + chunk * 8;
    aput[i] = lds + XB + (sub * 16 * NF + row) * 128 + (chunk ^ (row & 7)) * 16;
  }
  uint8_t *const xput = lds + (xsub * kTileM + xrow) * 128 + (chunk ^ (xrow & 7)) * 16;
  const int fp = wave % FP, h = wave / FP, frag = (((4 * h + g) & 7) ^ (r16 & 7)) * 16;  // this wave's 32 k
  const uint8_t *fa = lds + XB + ((h >> 1) * 16 * NF + 16 * FR * fp + r16) * 128 + frag, *fx = lds + ((h >> 1) * kTileM + r16) * 128 + frag;
  u32x4 xv[kDeep], av[kDeep][AP];
  f32x4 acc[FR];
#pragma unroll
  for (int f = 0; f < FR; ++f) acc[f] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](int buf) {
    wait_and_sync<63>();  // this stage is in LDS; loads stay under way
    const u32x4 x = *reinterpret_cast<const u32x4 *>(fx + buf);
#pragma unroll
    for (int f = 0; f < FR; ++f) acc[f] = mfma16x16x32(*reinterpret_cast<const u32x4 *>(fa + buf + f * 2048), x, acc[f]);
  };
  // whole stages
  const uint16_t *xp = xrowp + xk, *ap = av0;
  uint32_t aoff[AP];
#pragma unroll
  for (int i = 0; i < AP; ++i) aoff[i] = arow[i] + ak[i] * 2;
  auto load = [&](int d) {
    xv[d] = ld16(xp + d * KS);
#pragma unroll
    for (int i = 0; i < AP; ++i) av[d][i] = ld16_at(ap + d * KS, aoff[i]);
  };
  auto use = [&](int d) {
    *reinterpret_cast<u32x4 *>(xput + (d & 1) * STAGE) = xv[d];
#pragma unroll
    for (int i = 0; i < AP; ++i) *reinterpret_cast<u32x4 *>(aput[i] + (d & 1) * STAGE) = av[d][i];
  };
  // the last ones: pieces past K read the row's first and are zeroed on their way to LDS
  auto load_last = [&](int stage, int d) {
    const int k = stage * KS;
    xv[d] = ld16(xrowp + (k + xk < K ? k + xk : 0));
#pragma unroll
    for (int i = 0; i < AP; ++i) av[d][i] = ld16_at(av0, arow[i] + (k + ak[i] < K ? k + ak[i] : 0) * 2u);
  };
  auto use_last = [&](int stage, int d) {
    const int k = stage * KS;
    *reinterpret_cast<u32x4 *>(xput + (d & 1) * STAGE) = k + xk < K ? xv[d] : zero;
#pragma unroll
    for (int i = 0; i < AP; ++i) *reinterpret_cast<u32x4 *>(aput[i] + (d & 1) * STAGE) = k + ak[i] < K ? av[d][i] : zero;
  };
  const int groups = K / (KS * kDeep), stages = (K + KS - 1) / KS;  // groups of kDeep whole stages; all stages
  if (groups > 0) {
#pragma unroll
    for (int d = 0; d < kDeep; ++d) load(d);
    for (int i = 1; i < groups; ++i) {
      xp += KS * kDeep;
      ap += KS * kDeep;
#pragma unroll
      for (int d = 0; d < kDeep; ++d) {
        use(d);
        load(d);
        multiply((d & 1) * STAGE);
      }
    }
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      use(d);
      load_last(groups * kDeep + d, d);
      multiply((d & 1) * STAGE);
    }
  } else {
#pragma unroll
    for (int d = 0; d < kDeep; ++d) load_last(d, d);
  }
#pragma unroll
  for (int d = 0; d < kDeep; ++d) {
    if (groups * kDeep + d >= stages) break;
    use_last(groups * kDeep + d, d);
    multiply((d & 1) * STAGE);
  }
  f32x4 *part = reinterpret_cast<f32x4 *>(lds);  // [wave][FR][64]
  __syncthreads();
#pragma unroll
  for (int f = 0; f < FR; ++f) part[(wave * FR + f) * 64 + lane] = acc[f];
  __syncthreads();
  if (wave < NF) {  // row tile `wave`
    f32x4 sum = part[(wave / FR * FR + wave % FR) * 64 + lane];
#pragma unroll
    for (int q = 1; q < H; ++q) sum += part[((q * FP + wave / FR) * FR + wave % FR) * 64 + lane];
    const int j = j0 + 16 * wave + 4 * g, pitch = z_pitch(a.s.r);
    if (j < pitch - 8) {
      const float scale = a.scale[t.slot];
      f32x4 v;
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = j + k < t.rank ? sum[k] * scale : 0.f;
      store_parts(v, zs + r16 * pitch + j, kTileM * pitch);
    }
  }
  __syncthreads();
}

// z of a tile of up to NT tokens whose slot's rows are only read once: dot products
// in registers, no matrix cores (a tile of 16 tokens would use a sixteenth of them),
// no staging.  A wave takes 8 RS rows of V^T, 8 lanes a row, and a share of K; the
// lanes' and the waves' sums meet at the end.
__device__ __forceinline__ float dot8(u32x4 a, u32x4 b, float c) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, static_cast<uint32_t>(a[i])),
                                        __builtin_bit_cast(bf16x2, static_cast<uint32_t>(b[i])), c, false);
  return c;
}

template <int RS, int NT>
__device__ __forceinline__ void dot_z(const AdapterArgs &a, const Tile &t, const int *tok, int c, uint8_t *lds, uint16_t *zs) {
  constexpr int ROWS = 8 * RS, AHEAD = 4;  // steps of loads under way
  const int lane = threadIdx.x & 63, wave = keep(threadIdx.x >> 6), K = a.K;
  // groups of rows, and waves that share K for one
  const int need = (t.rank16 + ROWS - 1) / ROWS, groups = need <= 1 ? 1 : need <= 2 ? 2 : need <= 4 ? 4 : 8, share = kWaves / groups;
  const int group = wave % groups, part = wave / groups;
  const uint16_t *v0 = a.vt + ((static_cast<int64_t>(t.slot) * a.nchild + c) * a.s.r) * K;
  const int chunk = (lane & 7) * 8;
  uint32_t voff[RS];
#pragma unroll
  for (int s = 0; s < RS; ++s)  // (rows past the rank repeat the last and are masked)
    voff[s] = (static_cast<uint32_t>(min(group * ROWS + 8 * s + (lane >> 3), t.rank16 - 1)) * static_cast<uint32_t>(K) + chunk) * 2u;
  const uint16_t *xp[NT];
#pragma unroll
  for (int m = 0; m < NT; ++m) xp[m] = a.x + static_cast<int64_t>(keep(tok[m] < 0 ? tok[0] : tok[m])) * K;
  float acc[RS][NT];
#pragma unroll
  for (int s = 0; s < RS; ++s)
#pragma unroll
    for (int m = 0; m < NT; ++m) acc[s][m] = 0.f;
  const int stride = share * 64, whole = K / (stride * AHEAD);
  u32x4 v[AHEAD][RS], x[AHEAD][NT];
  int k = part * 64;
  for (int i = 0; i < whole; ++i) {
#pragma unroll
    for (int d = 0; d < AHEAD; ++d, k += stride) {
#pragma unroll
      for (int s = 0; s < RS; ++s) v[d][s] = ld16_at(v0 + k, voff[s]);
#pragma unroll
      for (int m = 0; m < NT; ++m) x[d][m] = ld16_at(xp[m] + k, chunk * 2u);
    }
#pragma unroll
    for (int d = 0; d < AHEAD; ++d)
#pragma unroll
      for (int s = 0; s < RS; ++s)
#pragma unroll
        for (int m = 0; m < NT; ++m) acc[s][m] = dot8(v[d][s], x[d][m], acc[s][m]);
  }
  const u32x4 zero{0u, 0u, 0u, 0u};
#pragma unroll
  for (int d = 0; d < AHEAD; ++d) {
    const bool in = k + d * stride + chunk < K;
    const uint32_t at = in ? (k + d * stride) * 2u : 0u;
#pragma unroll
    for (int s = 0; s < RS; ++s) v[d][s] = in ? ld16_at(v0, voff[s] + at) : zero;
#pragma unroll
    for (int m = 0; m < NT; ++m) x[d][m] = in ? ld16_at(xp[m], chunk * 2u + at) : zero;
  }
#pragma unroll
  for (int d = 0; d < AHEAD; ++d)
#pragma unroll
    for (int s = 0; s < RS; ++s)
#pragma unroll
      for (int m = 0; m < NT; ++m) acc[s][m] = dot8(v[d][s], x[d][m], acc[s][m]);
  float *sums = reinterpret_cast<float *>(lds);  // [wave][row][token]
#pragma unroll
  for (int s = 0; s < RS; ++s)
#pragma unroll
    for (int m = 0; m < NT; ++m) {
      float w = acc[s][m];
#pragma unroll
      for (int d = 1; d < 8; d <<= 1) w += __shfl_xor(w, d, 64);
      if ((lane & 7) == 0) sums[(wave * ROWS + 8 * s + (lane >> 3)) * NT + m] = w;
    }
  __syncthreads();
  const float scale = a.scale[t.slot];
  const int pitch = z_pitch(a.s.r);
  // four ranks of a token a thread
  for (int i = threadIdx.x; i < groups * (ROWS / 4) * NT; i += kThreads) {
    const int m = i % NT, j = i / NT * 4;  // j: row of V^T
    if (j >= t.rank16) continue;
    f32x4 v{0.f, 0.f, 0.f, 0.f};
    for (int q = 0; q < share; ++q)
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] += sums[((q * groups + j / ROWS) * ROWS + j % ROWS + k) * NT + m];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = j + k < t.rank ? v[k] * scale : 0.f;
    store_parts(v, zs + m * pitch + j, kTileM * pitch);
  }
  __syncthreads();
}

// y[t][n] = base[t][n] + sum_j c z[t][j] U_a[n][j] of the wave's turns, 64 n each.
// U, 32 ranks at a time, and the sums pass through a piece of LDS of the wave's own,
// so that U is read as rows and base and y as 128 bytes a token.  UNITS times 32 CW
// ranks hold the slot's (CW 0: one unit of 16, rows of 32 bytes); the loads of the
// next unit are under way while one is used, base's a turn ahead, and the first
// (of U up to 32 ranks) leave before form() makes z.  A child's last, partial 64 n are a turn of their own.
constexpr int kUPitch = 80, kOutPitch = 272, kWaveLds = 64 * kUPitch;  // bytes
static_assert(16 * kOutPitch <= kWaveLds, "the sums fit the piece");

template <int UNITS, int CW, bool ONCE>
struct RowWalk {
  static constexpr int CHUNKS = CW ? CW : 1, PER = CW ? 4 : 2, LOADS = PER * CHUNKS, ROWS = CW ? 16 : 32;
  static constexpr int COLS = CW ? 32 * CW * UNITS : 16;  // ranks it reads
  static constexpr bool EARLY = CW < 2;                   // (more would cost form() registers)
  const AdapterArgs &a;
  const Tile &t;
  const uint16_t *zs, *U;
  uint8_t *mine;
  int N, r, pitch, lane, r16, g, wave, urow, ucol;
  uint32_t uoff[PER];  // bytes from the first row of a turn
  // as rows: lane -> row lane / 8 (of 8) of base and y, 8 n from 8 (lane % 8) on
  int64_t at[2];
  bool has[2];

  __device__ __forceinline__ RowWalk(const AdapterArgs &a_, const Tile &t_, int c, const int *tok, const uint16_t *zs_, uint8_t *lds)
      : a(a_), t(t_), zs(zs_) {
    lane = threadIdx.x & 63;
    wave = keep(threadIdx.x >> 6);
    r16 = lane & 15;
    g = lane >> 4;
    urow = CW ? lane >> 2 : lane >> 1;
    ucol = CW ? (lane & 3) * 8 : (lane & 1) * 8;
    mine = lds + wave * kWaveLds;
    N = a.N[c];
    r = a.s.r;
    pitch = z_pitch(r);
    U = a.u + (static_cast<int64_t>(max(t.slot, 0)) * a.Ntot + a.n0[c]) * r;
#pragma unroll
    for (int q = 0; q < PER; ++q) uoff[q] = static_cast<uint32_t>((ROWS * q + urow) * r + ucol) * 2u;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int token = tok[8 * q + (lane >> 3)];
      has[q] = token >= 0;
      at[q] = static_cast<int64_t>(has[q] ? token : tok[0]) * a.Ntot + a.n0[c] + (lane & 7) * 8;
    }
  }
  // FULL: 64 rows exist, and where ranks are read past the room one more (what they
  // find, the next row's, is masked).  Otherwise rows past the last repeat it (not
  // stored) and ranks past the room the first.
  template <bool FULL>
  __device__ __forceinline__ void load_u(int nw, int unit, u32x4 (&o)[LOADS]) const {
    const uint16_t *p = U + static_cast<int64_t>(nw) * r;
#pragma unroll
    for (int ch = 0; ch < CHUNKS; ++ch)
#pragma unroll
      for (int q = 0; q < PER; ++q) {
        const int k0 = (unit * CHUNKS + ch) * 32;
        if constexpr (FULL)
          o[ch * PER + q] = ONCE ? ld16_once_at(p + k0, uoff[q]) : ld16_at(p + k0, uoff[q]);
        else
          o[ch * PER + q] = ld16(U + static_cast<int64_t>(min(nw + ROWS * q + urow, N - 1)) * r + (k0 + ucol < r ? k0 + ucol : 0));
      }
  }
  template <bool FULL>
  __device__ __forceinline__ void load_base(int nw, u32x4 (&o)[2]) const {
#pragma unroll
    for (int q = 0; q < 2; ++q)
      o[q] = FULL ? ld16_any(a.base + at[q] + nw) : load_some(a.base + at[q] + nw, N - (nw + (lane & 7) * 8));
  }
  template <bool FULL>
  __device__ __forceinline__ void store(int nw, const u32x4 (&o)[2]) const {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if (!has[q]) continue;
      if constexpr (FULL)
        st16_any(a.y + at[q] + nw, o[q]);
      else
        store_some(a.y + at[q] + nw, o[q], N - (nw + (lane & 7) * 8));
    }
  }
  // One turn: un holds its first unit of U, bn its base; afterwards both hold those
  // of the turn at `next`.
  template <bool FULL>
  __device__ __forceinline__ void turn(int nw, u32x4 (&un)[LOADS], u32x4 (&bn)[2], int next) const {
    const u32x4 zero{0u, 0u, 0u, 0u};
    f32x4 acc[4];
    u32x4 b[2];
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int q = 0; q < 2; ++q) b[q] = bn[q];
#pragma unroll
    for (int unit = 0; unit < UNITS; ++unit) {
#pragma unroll
      for (int ch = 0; ch < CHUNKS; ++ch) {
        const int k0 = (unit * CHUNKS + ch) * 32;
        if (k0 + (CW ? 32 : 16) > t.rank) {
#pragma unroll
          for (int q = 0; q < PER; ++q) un[ch * PER + q] = first_of_8(un[ch * PER + q], t.rank - (k0 + ucol));
        }
#pragma unroll
        for (int q = 0; q < PER; ++q) *reinterpret_cast<u32x4 *>(mine + (ROWS * q + urow) * kUPitch + ucol * 2) = un[ch * PER + q];
        if (ch == CHUNKS - 1) {
          load_u<FULL>(unit + 1 < UNITS ? nw : next, (unit + 1) % UNITS, un);
          if (unit == 0) load_base<FULL>(next, bn);
        }
        const bool in = CW || g < 2;  // (16 ranks: the other half of the contraction is zeros)
        u32x4 uv[4], zv[kParts];
#pragma unroll
        for (int p = 0; p < kParts; ++p) zv[p] = in ? ld16(zs + (p * kTileM + r16) * pitch + k0 + 8 * g) : zero;
#pragma unroll
        for (int j = 0; j < 4; ++j) uv[j] = in ? *reinterpret_cast<const u32x4 *>(mine + (16 * j + r16) * kUPitch + 16 * g) : zero;
#pragma unroll
        for (int p = 0; p < kParts; ++p)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[j] = mfma16x16x32(uv[j], zv[p], acc[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) *reinterpret_cast<f32x4 *>(mine + r16 * kOutPitch + (16 * j + 4 * g) * 4) = acc[j];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const f32x4 *o = reinterpret_cast<const f32x4 *>(mine + (8 * q + (lane >> 3)) * kOutPitch + (lane & 7) * 32);
      b[q] = add_8(b[q], o[0], o[1]);
    }
    store<FULL>(nw, b);
  }
  // Every wave calls form(), which has barriers.
  template <typename Z>
  __device__ __forceinline__ void run(int first, Z &&form) const {
    const int end = min(N, first + a.turns * kThreads), full = min(end, (N - (COLS > r ? 1 : 0)) / 64 * 64);
    int nw = first + wave * 64;
    u32x4 un[LOADS], bn[2];
    if (nw < full) {
      if (EARLY) load_u<true>(nw, 0, un);
      load_base<true>(nw, bn);
    }
    form();
    if (!EARLY && nw < full) load_u<true>(nw, 0, un);
    for (; nw < full; nw += kThreads) turn<true>(nw, un, bn, nw + kThreads < full ? nw + kThreads : nw);  // (the last loads itself again)
    if (nw >= end) return;
    load_u<false>(nw, 0, un);
    load_base<false>(nw, bn);
    turn<false>(nw, un, bn, nw);
  }
  // Tokens without an adapter.
  __device__ __forceinline__ void copy(int first) const {
    const int end = min(N, first + a.turns * kThreads);
    for (int nw = first + wave * 64; nw < end; nw += kThreads) {
      u32x4 b[2];
      if (nw + 64 <= N) {
        load_base<true>(nw, b);
        store<true>(nw, b);
      } else {
        load_base<false>(nw, b);
        store<false>(nw, b);
      }
    }
  }
};

// Child of workgroup blockIdx.y.
__device__ __forceinline__ int child_of(const AdapterArgs &a) {
  int c = 0;
#pragma unroll
  for (int i = 1; i < kMaxChildren; ++i)
    if (i < a.nchild && static_cast<int>(blockIdx.y) >= a.block0[i]) c = i;
  return c;
}

// ---- few tokens ------------------------------------------------------------------
constexpr int kRing = 2 * 24 * 1024;  // two stages of form_z<2>, the largest
static_assert(kWaves * kWaveLds <= kRing, "the waves' pieces lie over the stages");

// ROOM: the pool's rank rounded up to 16, 64 or 256 (what a slot of a larger rank
// needs costs the others registers; at 16 two workgroups fit a CU).  ONCE: much of
// U, rank 16 (whole lines a load), is read past the caches, in calls whose slots are many
// for their tokens (64 tokens of 57 adapters through 31B gate|up 30.5 -> 27.2 us; but 3200
// tokens of 4 through 4096 x 4096 17.8 -> 22.7, 400 of 64 at rank 64 34 -> 38) and there by
// tiles that are not full: a full one's slot is likely to have more, which read the same
// rows (1000 tokens in one of 64 slots of gate|up, past the caches 86, so 74; 64 of them 30
// and 27.8).
template <int ROOM, bool ONCE>
__global__ __launch_bounds__(kThreads, ROOM == 16 ? 4 : 2) void few_kernel(AdapterArgs a) {
  __shared__ int tok[kTileM];
  __shared__ __align__(16) uint8_t lds[kRing];
  extern __shared__ __align__(16) uint16_t zs[];  // [kParts][kTileM][pitch]
  Tile t;
  if (!get_tile<kTileM, kThreads>(a.s, blockIdx.x, t, tok)) return;
  const int c = child_of(a), first = (static_cast<int>(blockIdx.y) - a.block0[c]) * a.turns * kThreads;
  const auto form = [&] {
    // c z all zeros, which ranks past the slot's stay (barriers stand between this and the stores of z)
    for (int i = threadIdx.x; i < kParts * kTileM * z_pitch(a.s.r) / 8; i += kThreads) reinterpret_cast<u32x4 *>(zs)[i] = u32x4{0u, 0u, 0u, 0u};
    if (t.count == 1) {
      if (ROOM == 16 || t.rank16 == 16)
        dot_z<2, 1>(a, t, tok, c, lds, zs);
      else
        dot_z<4, 1>(a, t, tok, c, lds, zs);
      return;
    }
    for (int f = 0; f < t.rank16 / 16;) {
      const int live = t.rank16 / 16 - f;
      if (ROOM > 16 && live >= 3) {
        form_z<4>(a, t, tok, c, 16 * f, lds, zs);
        f += 4;
      } else if (ROOM > 16 && live == 2) {
        form_z<2>(a, t, tok, c, 16 * f, lds, zs);
        f += 2;
      } else {
        form_z<1>(a, t, tok, c, 16 * f, lds, zs);
        f += 1;
      }
    }
  };
  if (t.slot < 0)
    RowWalk<1, 0, ONCE>(a, t, c, tok, zs, lds).copy(first);
  else if (ONCE && t.count < kTileM)
    RowWalk<1, 0, ONCE>(a, t, c, tok, zs, lds).run(first, form);
  else if (ROOM == 16 || t.rank16 <= 16)
    RowWalk<1, 0, false>(a, t, c, tok, zs, lds).run(first, form);
  else if (t.rank16 <= 32)
    RowWalk<1, 1, false>(a, t, c, tok, zs, lds).run(first, form);
  else if (ROOM == 64 || t.rank16 <= 64)
    RowWalk<1, 2, false>(a, t, c, tok, zs, lds).run(first, form);
  else if (t.rank16 <= 128)
    RowWalk<2, 2, false>(a, t, c, tok, zs, lds).run(first, form);
  else
    RowWalk<4, 2, false>(a, t, c, tok, zs, lds).run(first, form);
}

// ---- many tokens -------------------------------------------------------------------
// z of a tile, a slice of K and 16 NF rows of V^T of all children.
template <int NF>
__global__ __launch_bounds__(kThreads, 4) void thin_kernel(ProjectArgs a) {
  __shared__ int tok[kM];
  __shared__ __align__(16) uint8_t lds[Stage<NF>::LDS];
  Tile t;
  if (!get_tile<kM>(a.s, blockIdx.x, t, tok) || t.slot < 0) return;
  project_z<NF, false>(a, t, tok, blockIdx.y, lds);
}

// 16 FRAGS of a tile's 64 tokens by 256 rows of U, 64 a wave, up to 32 CH ranks.  U
// passes through the wave's piece of LDS into registers, where it serves the tokens,
// 16 at a time; their sums pass through the piece again.  All of base is under way
// from the start.  c z comes from finish_kernel's pieces (PIECES), or each workgroup adds
// up z's slices into LDS.  (With the next 256 rows sent for while these are worked on,
// 2 to 6 times: registers for 2 workgroups on a CU, 4096 tokens through 5376 rows at
// rank 64 40 us, as it is 26 and 33.)
constexpr int kExpandWaves = 4;

template <int CH, int FRAGS, bool PIECES>
__global__ __launch_bounds__(kExpandWaves * 64) void expand_kernel(AdapterArgs a) {
  constexpr int MW = 16 * FRAGS;
  __shared__ int tok[kM];
  __shared__ __align__(16) uint8_t lds[kExpandWaves * kWaveLds];
  extern __shared__ __align__(16) uint16_t zs[];  // without pieces: [kParts][MW][pitch]
  Tile t;
  const int m0 = blockIdx.z * MW;
  if (!get_tile<kM>(a.s, blockIdx.x, t, tok) || m0 >= t.count) return;
  const int lane = threadIdx.x & 63, wave = keep(threadIdx.x >> 6), r16 = lane & 15, g = lane >> 4;
  const int c = child_of(a), N = a.N[c], r = a.s.r, pitch = z_pitch(r);
  const int nw = ((static_cast<int>(blockIdx.y) - a.block0[c]) * kExpandWaves + wave) * 64;
  const int chunks = t.slot >= 0 ? (t.rank16 + 31) / 32 : 0;
  uint8_t *const mine = lds + wave * kWaveLds;
  // as rows: lane -> row lane / 8 (of 8) of base and y, 8 n from 8 (lane % 8) on;
  // row lane / 4 (of 16) of U, 8 ranks from 8 (lane % 4) on
  const int orow = lane >> 3, ocol = (lane & 7) * 8, urow = lane >> 2, ucol = (lane & 3) * 8;
  const uint16_t *U = a.u + (static_cast<int64_t>(max(t.slot, 0)) * a.Ntot + a.n0[c]) * r;
  uint32_t uoff[4];  // bytes to the lanes' rows; rows past the last repeat it (not stored)
#pragma unroll
  for (int q = 0; q < 4; ++q) uoff[q] = static_cast<uint32_t>(max(0, min(16 * q + urow, N - 1 - nw)) * r) * 2u;
  const uint16_t *urows = U + static_cast<int64_t>(min(nw, N - 1)) * r;
  u32x4 un[4], u[CH][4];
  auto load_u = [&](int chunk) {  // (ranks past the room: the row's first, masked)
    const int k = chunk * 32 + ucol;
    const uint32_t kb = k < r ? k * 2u : 0u;
#pragma unroll
    for (int q = 0; q < 4; ++q) un[q] = ld16_at(urows, uoff[q] + kb);
  };
  const uint16_t *z0 = a.z + ((static_cast<int64_t>(blockIdx.x) * 4 + m0 / 16) * a.nchild + c) * a.RC * kPieces;
  u32x4 zn[kParts];
  auto load_z = [&](int i, int chunk) {
#pragma unroll
    for (int p = 0; p < kParts; ++p) zn[p] = ld16_at(z0 + ((i * a.nchild * a.RC + chunk) * kParts + p) * 512, lane * 16u);
  };
  u32x4 b[FRAGS][2];
  int64_t at[FRAGS][2];
#pragma unroll
  for (int i = 0; i < FRAGS; ++i)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int token = tok[m0 + 16 * i + 8 * q + orow];
      at[i][q] = static_cast<int64_t>(token < 0 ? tok[0] : token) * a.Ntot + a.n0[c] + nw + ocol;
    }
  if (chunks) load_u(0);
  const bool full = nw + 64 <= N;
  if (full) {
#pragma unroll
    for (int i = 0; i < FRAGS; ++i)
#pragma unroll
      for (int q = 0; q < 2; ++q) b[i][q] = PIECES ? ld16_any_once(a.base + at[i][q]) : ld16_any(a.base + at[i][q]);  // (31B o 59 -> 57 us)
  } else {
#pragma unroll
    for (int i = 0; i < FRAGS; ++i)
#pragma unroll
      for (int q = 0; q < 2; ++q) b[i][q] = load_some(a.base + at[i][q], N - (nw + ocol));
  }
  if (chunks) {
    if constexpr (PIECES) {
      load_z(0, 0);
    } else {
      const float scale = a.scale[t.slot];
      const int shift = 31 - __builtin_clz(pitch - 8) - 2;  // quads of a row, a power of two
      const int j = (threadIdx.x & ((1 << shift) - 1)) * 4;
      const float *row0 = a.P + (static_cast<int64_t>(blockIdx.x) * kM + m0) * a.R + c * r + j;
      for (int m = threadIdx.x >> shift; m < MW; m += (kExpandWaves * 64) >> shift) {
        f32x4 v{0.f, 0.f, 0.f, 0.f};
        if (m0 + m < t.count && j < t.rank16) {
          const float *p = row0 + m * a.R;
#pragma unroll 4
          for (int s = 0; s < a.slices; ++s) v += *reinterpret_cast<const f32x4 *>(p + s * a.rows * a.R);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = j + k < t.rank ? v[k] * scale : 0.f;
        store_parts(v, zs + m * pitch + j, MW * pitch);
      }
    }
#pragma unroll
    for (int ch = 0; ch < CH; ++ch) {
      if (ch >= chunks) break;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<u32x4 *>(mine + (16 * q + urow) * kUPitch + ucol * 2) = first_of_8(un[q], t.rank - (ch * 32 + ucol));
      if (ch + 1 < CH) load_u(min(ch + 1, chunks - 1));
#pragma unroll
      for (int j = 0; j < 4; ++j) u[ch][j] = *reinterpret_cast<const u32x4 *>(mine + (16 * j + r16) * kUPitch + 16 * g);
    }
    if constexpr (!PIECES) __syncthreads();
  }
  if (nw >= N) return;
#pragma unroll
  for (int i = 0; i < FRAGS; ++i) {
    if (m0 + 16 * i >= t.count) break;
    if (chunks) {
      f32x4 acc[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ch = 0; ch < CH; ++ch) {
        if (ch >= chunks) break;
        u32x4 z[kParts];
        if constexpr (PIECES) {
#pragma unroll
          for (int p = 0; p < kParts; ++p) z[p] = zn[p];
          if (ch + 1 < CH && ch + 1 < chunks)
            load_z(i, ch + 1);
          else
            load_z(min(i + 1, FRAGS - 1), 0);
        } else {
#pragma unroll
          for (int p = 0; p < kParts; ++p) z[p] = ld16(zs + (p * MW + 16 * i + r16) * pitch + 32 * ch + 8 * g);
        }
#pragma unroll
        for (int p = 0; p < kParts; ++p)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[j] = mfma16x16x32(u[ch][j], z[p], acc[j]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) *reinterpret_cast<f32x4 *>(mine + r16 * kOutPitch + (16 * j + 4 * g) * 4) = acc[j];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const f32x4 *o = reinterpret_cast<const f32x4 *>(mine + (8 * q + orow) * kOutPitch + ocol * 4);
        b[i][q] = add_8(b[i][q], o[0], o[1]);
      }
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if (m0 + 16 * i + 8 * q + orow >= t.count) continue;
      if (full)
        st16_any(a.y + at[i][q], b[i][q]);
      else
        store_some(a.y + at[i][q], b[i][q], N - (nw + ocol));
    }
  }
}

// ---- plan ----------------------------------------------------------------------
constexpr int kMaxSlices = 6;

struct Plan {
  bool few;           // few_kernel
  bool grouped;       // group_kernel first
  int tiles;          // most tiles there can be
  int blocks, turns;  // workgroups along the children's rows, turns of a wave
  int across;         // rows of a workgroup
  int NF, zgroups, slices, per, frags, RC;
  bool pieces;
  int64_t rows;
  size_t perm_at, z_at, p_at, bytes;
};

// Which launches: few_kernel alone, few_kernel over tiles of 16 that group_kernel has
// made, or tiles of 64 with z in a launch of its own.  The least of three estimates, in ns:
//   few_kernel    5000, z once a workgroup (31 products of V^T a ns, 46 for one token), 1000
//                 for 512 rows of U a CU (more where a higher rank leaves it fewer waves),
//                 counted for as many tiles as there can be, base and y at 6 TB/s, x at 5
//   group_kernel  5000
//   the others    15000, x and V^T, expand_kernel's workgroups (900 in 4300 ns) or base
//                 and y, U, and 5000 for finish_kernel
// Kernels' times in us, in that order (most within 20% of the estimates; over 60 drawn calls
// the choice is 2% slower than the best of the three, in 10 of them more than 5%, at worst 32%;
// tiles of 64 that are mostly part-filled are counted too low: the third figure of 1600):
//   333 tokens of 1160 -> 1001, rank 32            9.6  12.5  14.8
//   64 tokens of 57 adapters, 31B gate|up, rank 16  28    33    66;  400: 81, 54, 72;  1600: -, 106, 124
//   4096 -> 4096, rank 16, 200 tokens 13.8, 12.8, 15.2;  3200: -, 25, 34
//   31B gate|up, 8 adapters, 400 tokens -, 27, 42;  800: -, 59, 53;  3200: -, 164, 151
//   4096 -> 4096, rank 128, 200 tokens 37, 31, 23;  8192 -> 5376, rank 64, 400: 36, 30, 27
enum class Form { kAlone, kGrouped16, kGrouped64 };

Form fastest_form(const AdapterPool &p, int T) {
  int64_t turns = 0, blocks = 0;
  for (int c = 0; c < p.nchild; ++c) {
    turns += (p.N[c] + kThreads - 1) / kThreads;
    blocks += (p.N[c] + kExpandWaves * 64 - 1) / (kExpandWaves * 64);
  }
  const int64_t K = p.K, N = p.Ntot, live = std::min(p.n, T);
  const int64_t x = T * K / 2500, out = T * N / 1250;  // 2 and 4 bytes at 5 TB/s
  const auto few = [&](int64_t tiles) {
    return 5000 + K * p.r / (T == 1 ? 46 : 31) + turns * tiles * (p.r <= 32 ? 950 : p.r <= 64 ? 1500 : 2400) / kCUs + out * 4 / 5 + x;
  };
  const int64_t alone = few(T), grouped16 = 5000 + few(std::min(T, p.n + 1 + T / kTileM));
  const int64_t busy = (T + kM - 1) / kM, tiles = std::min(T, p.n + 1 + T / kM);
  const int64_t grouped64 = 14500 + x * 13 / 10 + live * p.nchild * p.r * K / 5000 + live * N * p.r / 5000 +
                            std::max(tiles * blocks * 48 / 10, out * 11 / 10) + (blocks >= 16 && blocks * busy >= 2 * kCUs ? 5000 : 0);
  if (T <= kThreads && alone <= std::min(grouped16, grouped64)) return Form::kAlone;
  return grouped16 <= grouped64 ? Form::kGrouped16 : Form::kGrouped64;
}

Plan make_plan(const AdapterPool &p, int T) {
  Plan q{};
  const Form form = fastest_form(p, T);
  q.few = form != Form::kGrouped64;
  q.grouped = form != Form::kAlone;
  q.turns = 1;
  auto count_blocks = [&](int across) {
    q.across = across;
    q.blocks = 0;
    for (int c = 0; c < p.nchild; ++c) q.blocks += (p.N[c] + across - 1) / across;
  };
  if (q.few) {
    // (a token's workgroups on one XCD: they read the same V^T)
    const int most = q.grouped ? std::min(T, p.n + 1 + T / kTileM) : T;
    q.tiles = most < 8 && !q.grouped ? most : tile_places(most);
    // A workgroup for each CU, or two where they fit and have enough to walk over: 4
    // tokens through 2 x 21504 rows at rank 16 in 168 workgroups 7.3 us, in 336 10.0;
    // 64 tokens in 228 workgroups 30.0, in 456 27.8.
    count_blocks(kThreads);
    const int64_t all = static_cast<int64_t>(q.blocks) * most;
    q.turns = static_cast<int>((all + kCUs - 1) / kCUs);
    if (p.r == 16 && q.turns > 8) q.turns = static_cast<int>((all + 2 * kCUs - 1) / (2 * kCUs));
    count_blocks(kThreads * q.turns);
    q.perm_at = align256(sizeof(int4) * q.tiles);  // (the tiles come first)
    q.bytes = q.grouped ? q.perm_at + align256(sizeof(int32_t) * q.tiles * kTileM) : 256;
    return q;
  }
  count_blocks(kExpandWaves * 64);
  q.tiles = tile_places(T / kM + std::min(p.n + 1, T));
  const int busy = (T + kM - 1) / kM, row_tiles = p.nchild * p.r / 16;
  q.NF = row_tiles >= 3 ? 4 : row_tiles;
  q.zgroups = (row_tiles + q.NF - 1) / q.NF;
  // Four fragments of tokens serve a workgroup's rows of U, one where the tiles are too
  // few to fill the CUs (333 tokens through 1001 rows: 5.1 us, with four 10.5).
  q.frags = static_cast<int64_t>(q.blocks) * busy >= 2 * kCUs ? 4 : 1;
  cut_slices(p.K, q.NF == 4 ? 64 : 128, kDeep, busy * q.zgroups, kMaxSlices, q.slices, q.per);
  q.RC = (p.r + 31) / 32;
  // Where many workgroups would add up the same slices, finish_kernel does, once (4096
  // tokens, 2 x 21504 rows at rank 16: 173 -> 152 us and 5 for it; 5376 rows at rank 64, 21
  // workgroups: 33 -> 26 and 6; 1536 rows of 2048 tokens: 6.9 -> 5.1 and 4).
  q.pieces = q.frags == 4 && q.slices > 1 && q.blocks >= 16;
  q.rows = static_cast<int64_t>(q.tiles) * kM;
  q.perm_at = align256(sizeof(int4) * q.tiles);  // the tiles come first
  q.z_at = q.perm_at + align256(sizeof(int32_t) * q.rows);
  q.p_at = q.z_at + (q.pieces ? align256(kParts * sizeof(uint16_t) * q.rows * p.nchild * q.RC * 32) : 0);
  q.bytes = q.p_at + align256(sizeof(float) * q.slices * q.rows * p.nchild * p.r);
  return q;
}

template <int CH, int FRAGS, bool PIECES>
hipError_t launch_expand(const AdapterArgs &a, const Plan &q, hipStream_t stream) {
  constexpr size_t lds = PIECES ? 0 : sizeof(uint16_t) * kParts * 16 * FRAGS * z_pitch(32 * CH);
  const hipError_t e = ensure_lds<expand_kernel<CH, FRAGS, PIECES>>(lds);
  if (e != hipSuccess) return e;
  expand_kernel<CH, FRAGS, PIECES><<<dim3(q.tiles, q.blocks, 4 / FRAGS), kExpandWaves * 64, lds, stream>>>(a);
  return hipGetLastError();
}

template <int FRAGS, bool PIECES>
hipError_t launch_expand(const AdapterArgs &a, const Plan &q, hipStream_t stream) {
  if (a.s.r <= 32) return launch_expand<1, FRAGS, PIECES>(a, q, stream);
  if (a.s.r <= 64) return launch_expand<2, FRAGS, PIECES>(a, q, stream);
  if (a.s.r <= 128) return launch_expand<4, FRAGS, PIECES>(a, q, stream);
  return launch_expand<8, FRAGS, PIECES>(a, q, stream);
}

}  // namespace

size_t adapters_workspace_bytes(const AdapterPool &p, int T) { return T > 0 ? make_plan(p, T).bytes : 256; }

hipError_t launch_adapters(const AdapterPool &p, const uint16_t *x, const int32_t *index, int T, const uint16_t *base,
                           uint16_t *y, void *ws, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  const Plan q = make_plan(p, T);
  AdapterArgs a{};
  a.s.index = index;
  a.s.rank = p.rank;
  a.s.T = T;
  a.s.n = p.n;
  a.s.r = p.r;
  a.s.copies = base != y;
  a.x = x;
  a.vt = p.vt;
  a.u = p.u;
  a.scale = p.scale;
  a.base = base;
  a.y = y;
  a.R = p.nchild * p.r;
  a.K = p.K;
  a.Ntot = p.Ntot;
  a.nchild = p.nchild;
  a.turns = q.turns;
  for (int c = 0, n0 = 0, b0 = 0; c < p.nchild; ++c) {
    a.N[c] = p.N[c];
    a.n0[c] = n0;
    a.block0[c] = b0;
    n0 += p.N[c];
    b0 += (p.N[c] + q.across - 1) / q.across;
  }
  uint8_t *w = static_cast<uint8_t *>(ws);
  if (q.grouped) {
    GroupArgs g{};
    a.s.max_tiles = q.tiles;
    g.s = a.s;
    g.tiles = reinterpret_cast<int4 *>(w);
    g.perm = reinterpret_cast<int32_t *>(w + q.perm_at);
    const hipError_t e = q.few ? launch_group<kTileM>(g, stream) : launch_group<kM>(g, stream);
    if (e != hipSuccess) return e;
    a.s.tiles = g.tiles;
    a.s.perm = g.perm;
  }
  if (q.few) {
    const dim3 grid(q.tiles, q.blocks);
    const size_t lds = sizeof(uint16_t) * kParts * kTileM * z_pitch(p.r);
    const bool once = p.r == 16 && T <= kTileM * p.n && static_cast<int64_t>(std::min(p.n, T)) * p.Ntot * 32 >= 32 << 20;
    if (once)
      few_kernel<16, true><<<grid, kThreads, lds, stream>>>(a);
    else if (p.r == 16)
      few_kernel<16, false><<<grid, kThreads, lds, stream>>>(a);
    else if (p.r <= 64)
      few_kernel<64, false><<<grid, kThreads, lds, stream>>>(a);
    else
      few_kernel<256, false><<<grid, kThreads, lds, stream>>>(a);
    return hipGetLastError();
  }
  hipError_t e = hipSuccess;
  ProjectArgs z{};
  z.s = a.s;
  z.xb = x;
  z.vt = p.vt;
  z.K = p.K;
  z.nchild = p.nchild;
  z.R = a.R;
  z.rows = q.rows;
  z.zgroups = q.zgroups;
  z.zslices = q.slices;
  z.zper = q.per;
  z.Pz = reinterpret_cast<float *>(w + q.p_at);
  const dim3 thin(q.tiles, q.zgroups * q.slices);
  if (q.NF == 1)
    thin_kernel<1><<<thin, kThreads, 0, stream>>>(z);
  else if (q.NF == 2)
    thin_kernel<2><<<thin, kThreads, 0, stream>>>(z);
  else
    thin_kernel<4><<<thin, kThreads, 0, stream>>>(z);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  a.P = z.Pz;
  a.rows = q.rows;
  a.slices = q.slices;
  if (q.pieces) {
    FinishArgs f{};
    f.s = a.s;
    f.P[0] = z.Pz;
    f.slices[0] = q.slices;
    f.R = a.R;
    f.rows = q.rows;
    f.out.scale = p.scale;
    f.out.rows[0] = reinterpret_cast<uint16_t *>(w + q.z_at);
    f.out.RT = a.R / 16;
    f.out.nchild = p.nchild;
    f.out.RC = q.RC;
    finish_kernel<<<dim3(q.tiles, p.nchild * q.RC), 256, 0, stream>>>(f);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    a.z = f.out.rows[0];
    a.RC = q.RC;
    return launch_expand<4, true>(a, q, stream);
  }
  return q.frags == 1 ? launch_expand<1, false>(a, q, stream) : launch_expand<4, false>(a, q, stream);
}

}  // namespace wl
