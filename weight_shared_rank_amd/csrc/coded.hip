// 8-bit coded operands and their product.
//
// Coding.  An operand is cut into blocks along K, 128 elements of one token
// row for activations and 128 rows x 128 k for weights (the last ones
// short).  A block stores E4M3 codes and one power-of-two scale 2^e: e is the
// smallest exponent with max|x| <= 448 * 2^e, at least -118, and 0 for a block
// of zeros; a code is E4M3(x * 2^-e), nearest even.  x * 2^-e is exact and
// never exceeds 448, so each code is off by at most half an E4M3 step.
// Because the scale is a power of two, code * 2^e is a bf16 value exactly
// (4 significant bits; the bound on e keeps its smallest step, 2^-127, a
// multiple of bf16's 2^-133, and codes stop at 240 where 256 * 2^120 would
// leave its range), and the matrix cores apply it themselves: the
// scale byte e + 127 is their E8M0 block scale.  Elements that are not finite
// get the NaN code and do not count in a block's maximum.
//
// Layout of a coded operand [R, K] (Kq = K rounded up to 128, nb = Kq / 128):
//   codes  [R][Kq] bytes, row-major; codes at k >= K are zero
//   scales [nb][Rp] bytes, k-block-major (activations: one byte per token,
//          Rp = R rounded up to 16; weights: one per 128 rows, Rp = that
//          count rounded up to 4), at the next 256-byte offset.  A k step of
//          the product then reads the scales of a tile's rows as one run.
//
// Product  y[t][n] = sum_b 2^(ex[t,b] + ew[n/128,b]) sum_{k in b} cx[t,k] cw[n,k]
// on v_mfma_scale_f32_16x16x128_f8f6f4 (one instruction per k block and 16 x
// 16 outputs; both scales enter the instruction), y rounded to bf16 once.  The
// instruction adds the products of 8 consecutive k on a fixed-point grid 13
// binary places below the largest one's exponent (measured; a GPU test pins
// it), and those sums and the accumulator are fp32: on normal data the grid
// costs 1e-4 of a result, against the 2e-3 of rounding y to bf16.  The bf16
// instructions would add exactly at half the rate.
#include <algorithm>

#include "coded.h"
#include "common.h"
#include "lds_dma.h"
#include "training.h"

namespace wl {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kBlk = kCodeBlock;
constexpr int kCUs = 256;

// D += 2^(sa-127) 2^(sb-127) A B for a 16 x 16 tile over 128 k of E4M3 codes.
// Lane l supplies 32 codes of A row l & 15 and of B column l & 15 (any
// assignment of k to lane groups and bytes works as long as A and B share
// it); every lane passes the scale byte of its own row or column, the same in
// the four lane groups because a scale covers all 128 k.  D as mfma16x16x32.
__device__ __forceinline__ f32x4 mfma_coded(i32x8 a, i32x8 b, f32x4 c, int sa, int sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, sa, 0, sb);
}

__device__ __forceinline__ i32x8 join(u32x4 lo, u32x4 hi) {
  return __builtin_shufflevector(__builtin_bit_cast(i32x4, lo), __builtin_bit_cast(i32x4, hi), 0, 1, 2, 3, 4, 5, 6, 7);
}

// Largest |element| of 8 bf16 as its bit pattern (bf16 magnitudes order as
// integers); infinities and NaN count as zero.
__device__ __forceinline__ uint32_t amax_bits(u32x4 v) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = v[i] & 0x7fffu, hi = (v[i] >> 16) & 0x7fffu;
    m = max(m, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
  }
  return m;
}

// Smallest e with m <= 448 * 2^e = 1.75 * 2^(e + 8), at least -118; 0 for m = 0.
__device__ __forceinline__ int block_exponent(uint32_t m) {
  if (m == 0) return 0;
  const int e = static_cast<int>(m >> 7) - 127 - 8 + ((m & 0x7fu) > 0x60u ? 1 : 0);
  return max(e, -118);
}

// 8 bf16 -> 8 E4M3 codes of x * 2^-e; at the largest exponent magnitudes stop
// at 240, the next code's 256 * 2^120 being past bf16's range.
__device__ __forceinline__ u32x2 code8(u32x4 v, int e) {
  const float f = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  u32x2 o;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float x[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      x[2 * i] = __uint_as_float(v[2 * h + i] << 16);
      x[2 * i + 1] = __uint_as_float(v[2 * h + i] & 0xffff0000u);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[i] = fabsf(x[i]) < __builtin_inff() ? x[i] * f : __builtin_nanf("");
    if (e == 120)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (fabsf(x[i]) > 240.f) x[i] = copysignf(240.f, x[i]);
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], w, true);
    o[h] = static_cast<uint32_t>(w);
  }
  return o;
}

// Activations: a workgroup codes 16 tokens x kEncBlocks k blocks; 16 lanes
// share a block (8 elements each), so the reads and the stores of a wave are
// whole 256- and 128-byte runs and the maximum is four lane exchanges.  The
// scales of a k block's 16 tokens leave as one 16-byte run.
constexpr int kEncBlocks = 4;

__global__ __launch_bounds__(256) void encode_act_kernel(const uint16_t *x, int T, int K, int nb, uint8_t *codes,
                                                         uint8_t *scales, int ldsc) {
  const int l = threadIdx.x & 15, row = threadIdx.x >> 4;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * 16, tok = t0 + row;
  const int b0 = blockIdx.y * kEncBlocks;
  const int Kq = nb * kBlk;
  __shared__ __align__(16) uint8_t sc[kEncBlocks][16];
  u32x4 v[kEncBlocks];
#pragma unroll
  for (int i = 0; i < kEncBlocks; ++i) {
    const int k = (b0 + i) * kBlk + l * 8;
    v[i] = u32x4{0u, 0u, 0u, 0u};
    if (tok < T && k < K) v[i] = ld16(x + tok * K + k);
  }
#pragma unroll
  for (int i = 0; i < kEncBlocks; ++i) {
    uint32_t m = amax_bits(v[i]);
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), d, 16)));
    const int e = block_exponent(m);
    if (l == 0) sc[i][row] = static_cast<uint8_t>(e + 127);
    if (tok < T && b0 + i < nb)
      *reinterpret_cast<u32x2 *>(codes + tok * Kq + (b0 + i) * kBlk + l * 8) = code8(v[i], e);
  }
  __syncthreads();
  if (threadIdx.x < 4 * kEncBlocks) {
    const int i = threadIdx.x >> 2, w = threadIdx.x & 3;
    if (b0 + i < nb)
      reinterpret_cast<uint32_t *>(scales + static_cast<int64_t>(b0 + i) * ldsc + t0)[w] =
          reinterpret_cast<const uint32_t *>(sc[i])[w];
  }
}

// Weights: one workgroup per 128 x 128 block, held in registers between the
// maximum and the coding (the block is read once).
__global__ __launch_bounds__(256) void encode_weight_kernel(const uint16_t *w, int N, int K, int nb, uint8_t *codes,
                                                            uint8_t *scales, int ldsc) {
  const int l = threadIdx.x & 15, r0 = threadIdx.x >> 4;
  const int kb = blockIdx.x, k = kb * kBlk + l * 8;
  const int Kq = nb * kBlk;
  __shared__ uint32_t part[4];
  u32x4 v[8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t row = static_cast<int64_t>(blockIdx.y) * kBlk + i * 16 + r0;
    v[i] = u32x4{0u, 0u, 0u, 0u};
    if (row < N && k < K) v[i] = ld16(w + row * K + k);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, amax_bits(v[i]));
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), d, 64)));
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
  __syncthreads();
  m = max(max(part[0], part[1]), max(part[2], part[3]));
  const int e = block_exponent(m);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t row = static_cast<int64_t>(blockIdx.y) * kBlk + i * 16 + r0;
    if (row < N) *reinterpret_cast<u32x2 *>(codes + row * Kq + k) = code8(v[i], e);
  }
  if (threadIdx.x == 0) scales[static_cast<int64_t>(kb) * ldsc + blockIdx.y] = static_cast<uint8_t>(e + 127);
  // the pad bytes of a k block's run (up to 3) read as scale 1
  if (blockIdx.y == gridDim.y - 1 && threadIdx.x > 0 && blockIdx.y + threadIdx.x < static_cast<unsigned>(ldsc))
    scales[static_cast<int64_t>(kb) * ldsc + blockIdx.y + threadIdx.x] = 127;
}

// x[t][k] = code * 2^e as bf16 (exact), 8 elements per thread.
__global__ __launch_bounds__(256) void expand_act_kernel(CodedView c, uint16_t *x, int K) {
  const int k = (blockIdx.y * 256 + threadIdx.x) * 8;
  const int64_t tok = blockIdx.x;
  if (k >= K) return;
  *reinterpret_cast<u32x4 *>(x + tok * K + k) = expand8(c, tok, k);
}

struct CodedArgs {
  const uint8_t *W, *sw;  // weight codes [N][K], scales [nb][ldsw]
  const uint8_t *X, *sx;  // activation codes [T][K], scales [nb][ldsx]
  const uint16_t *x;      // coding fused: bf16 [T][Kx], coded into X and sx
  int32_t Kx;
  uint16_t *Y;            // [T][N]
  float *P;               // K-split partials [ksplit][T][ldp] (null: none)
  int32_t ldsw, ldsx, ldp;
  int32_t N, T, K, nb;    // K = nb * 128
  int32_t nM, nT, ksplit, steps_per_slice;
  int32_t rows;           // streaming: weight rows of a workgroup
};

// ---- few tokens (T <= 16): weight streaming -----------------------------------
// The weights go straight from HBM to registers as the A operand, each row
// read in 128-byte blocks by four lanes; the tokens' codes are the B operand
// (lanes past the last token repeat the first: their columns are not stored).
// Bound by reading N K bytes.  21504 x 5376 at T = 1, calls in a graph: 20.3 us
// over one weight again and again, 116 MB that stay in the 256 MB Infinity
// Cache (5.7 TB/s; 20.5 us for loads alone), 23.9 us where six weights take
// turns and each comes from HBM (4.8 TB/s).

// A workgroup's up to 16 rows over the whole K; its 16 waves take pairs of
// blocks in turn, so that neighbouring waves read neighbouring runs of the same
// rows, and their sums meet in LDS in wave order.  a.rows <= 16 is chosen so
// that the workgroups are a multiple of the CUs (21504 rows: 14, 21.5 us
// against 22.5 at 16; 8 waves of 4 blocks 23.5; loads one pair ahead 35).
//
// FUSE (T <= kFuseT): x comes as bf16 and every wave codes the blocks it needs,
// 16 lanes to a block as encode_act_kernel, through its part of LDS; workgroup
// 0 also writes the coded buffer.  It saves the coding launch and the x loads'
// turn (several weights in turn, 21504 x 5376 at T = 1: 25.2 us against 24.9 + 4
// for the two launches, 4096 x 1152: 3.5 against 3.0 + 3).  Two blocks a lane group, which would take
// 4 tokens, spills at 8 waves per SIMD: 47 us.
constexpr int kStreamWaves = 16, kStreamPair = 2;
constexpr int kFuseT = 4 / kStreamPair;  // a wave's 4 groups of 16 lanes code a pair's blocks at once

template <bool FUSE>
__global__ __launch_bounds__(kStreamWaves * 64) __attribute__((amdgpu_waves_per_eu(8, 8))) void
coded_stream_kernel(CodedArgs a) {
  constexpr int NW = kStreamWaves, S = kStreamPair;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r16 = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * a.rows;
  const bool live = r16 < a.rows && n0 + r16 < a.N;
  const int row = live ? n0 + r16 : n0;
  const uint8_t *wp = a.W + static_cast<int64_t>(row) * a.K + g * 16;
  const uint8_t *swp = a.sw + row / kBlk;
  const int tok = r16 < a.T ? r16 : 0;
  const uint8_t *xp = a.X + static_cast<int64_t>(tok) * a.K + g * 16;
  const uint8_t *sxp = a.sx + tok;
  __shared__ __align__(16) uint8_t xc[FUSE ? NW : 1][kFuseT][S * kBlk];
  __shared__ uint8_t xs[FUSE ? NW : 1][kFuseT][S];
  f32x4 acc{0.f, 0.f, 0.f, 0.f};
  const u32x4 zero{0u, 0u, 0u, 0u};
  for (int b = wave * S; b < a.nb; b += NW * S) {
    u32x4 w[S][2], x[S][2];
    int sw[S], sx[S];
    // FUSE: 16 lanes to a block (token t, block i of the pair), 8 elements each
    const int t = g / S, ti = g % S;
    u32x4 v = zero;
    if constexpr (FUSE) {
      const int k = (b + ti) * kBlk + r16 * 8;
      if (t < a.T && k < a.Kx) v = ld16(a.x + static_cast<int64_t>(t) * a.Kx + k);
    }
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int kb = min(b + i, a.nb - 1);
      w[i][0] = w[i][1] = zero;
      if (live) {
        w[i][0] = *reinterpret_cast<const u32x4 *>(wp + kb * kBlk);
        w[i][1] = *reinterpret_cast<const u32x4 *>(wp + kb * kBlk + 64);
      }
      sw[i] = swp[static_cast<int64_t>(kb) * a.ldsw];
    }
    if constexpr (FUSE) {
      asm volatile("" ::: "memory");
      uint32_t m = amax_bits(v);
#pragma unroll
      for (int d = 1; d < 16; d <<= 1) m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), d, 16)));
      const int e = block_exponent(m);
      const u32x2 c = code8(v, e);
      *reinterpret_cast<u32x2 *>(&xc[wave][t][ti * kBlk + r16 * 8]) = c;
      if (r16 == 0) xs[wave][t][ti] = static_cast<uint8_t>(e + 127);
      if (blockIdx.x == 0 && b + ti < a.nb) {
        if (t < a.T)
          *reinterpret_cast<u32x2 *>(const_cast<uint8_t *>(a.X) + static_cast<int64_t>(t) * a.K + (b + ti) * kBlk + r16 * 8) = c;
        // a block's 16 scale bytes: the tokens', and 127 behind them
        uint8_t *so = const_cast<uint8_t *>(a.sx) + static_cast<int64_t>(b + ti) * a.ldsx;
        if (r16 == 0 && t < a.T) so[t] = static_cast<uint8_t>(e + 127);
        if (t == 0 && r16 >= a.T) so[r16] = 127;
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
      for (int i = 0; i < S; ++i) {
        x[i][0] = *reinterpret_cast<const u32x4 *>(&xc[wave][tok][i * kBlk + g * 16]);
        x[i][1] = *reinterpret_cast<const u32x4 *>(&xc[wave][tok][i * kBlk + g * 16 + 64]);
        sx[i] = xs[wave][tok][i];  // a block past the end is zeros
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    } else {
#pragma unroll
      for (int i = 0; i < S; ++i) {
        const int kb = min(b + i, a.nb - 1);
        const bool in = b + i < a.nb;  // steps past the end multiply zeros
        x[i][0] = in ? *reinterpret_cast<const u32x4 *>(xp + kb * kBlk) : zero;
        x[i][1] = in ? *reinterpret_cast<const u32x4 *>(xp + kb * kBlk + 64) : zero;
        sx[i] = sxp[static_cast<int64_t>(kb) * a.ldsx];
      }
    }
#pragma unroll
    for (int i = 0; i < S; ++i)
      acc = mfma_coded(join(w[i][0], w[i][1]), join(x[i][0], x[i][1]), acc, sw[i], sx[i]);
  }
  __shared__ float part[NW][16][16];  // [wave][token][row]
  *reinterpret_cast<f32x4 *>(&part[wave][r16][g * 4]) = acc;
  __syncthreads();
  if (threadIdx.x < 256) {
    const int t = threadIdx.x >> 4, r = threadIdx.x & 15;
    if (t < a.T && r < a.rows && n0 + r < a.N) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < NW; ++i) s += part[i][t][r];
      a.Y[static_cast<int64_t>(t) * a.N + n0 + r] = f32_to_bf16(s);
    }
  }
}

// Several tokens: every code of x is then real, and a wave that loads 16 x 128
// of them per 16 x 128 weights is bound by the loads from L2, not HBM (5376 x
// 21504 at T = 16: 42 us).  Here a wave multiplies four 16-row tiles by each x
// fragment, a workgroup's 8 waves take blocks in turn, and K is cut into
// slices so that the workgroups fill the CUs; their partial sums go through
// coded_sum_kernel (252 workgroups of 3 slices and the sum: 26.4 us).  The
// scale bytes of a slice (at most kStreamSlice blocks) wait in LDS.
constexpr int kWideRows = 64, kWideWaves = 8, kStreamSlice = 256;
constexpr int kNarrowT = 4;  // up to here the one-tile kernel, which needs no workspace

__global__ __launch_bounds__(kWideWaves * 64) void coded_wide_kernel(CodedArgs a) {
  constexpr int NW = kWideWaves, RT = kWideRows / 16;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r16 = lane & 15, g = lane >> 4;
  const int tile = blockIdx.x / a.ksplit, sl = blockIdx.x % a.ksplit;
  const int b0 = min(a.nb, sl * a.steps_per_slice), b1 = min(a.nb, b0 + a.steps_per_slice);
  const int n0 = tile * kWideRows;  // 64 rows lie in one 128-row scale block
  __shared__ __align__(16) uint8_t xs[kStreamSlice * 16];
  __shared__ uint8_t ws[kStreamSlice];
  for (int i = threadIdx.x; i < b1 - b0; i += NW * 64) {
    *reinterpret_cast<u32x4 *>(xs + i * 16) = *reinterpret_cast<const u32x4 *>(a.sx + static_cast<int64_t>(b0 + i) * a.ldsx);
    ws[i] = a.sw[static_cast<int64_t>(b0 + i) * a.ldsw + n0 / kBlk];
  }
  __syncthreads();
  const uint8_t *wp[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
    wp[r] = a.W + static_cast<int64_t>(min(n0 + r * 16 + r16, a.N - 1)) * a.K + g * 16;
  const int tok = r16 < a.T ? r16 : 0;
  const uint8_t *xp = a.X + static_cast<int64_t>(tok) * a.K + g * 16;
  f32x4 acc[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) acc[r] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int b = b0 + wave; b < b1; b += NW) {
    u32x4 w[RT][2], x[2];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      w[r][0] = *reinterpret_cast<const u32x4 *>(wp[r] + b * kBlk);
      w[r][1] = *reinterpret_cast<const u32x4 *>(wp[r] + b * kBlk + 64);
    }
    x[0] = *reinterpret_cast<const u32x4 *>(xp + b * kBlk);
    x[1] = *reinterpret_cast<const u32x4 *>(xp + b * kBlk + 64);
    const int sx = xs[(b - b0) * 16 + tok], sw = ws[b - b0];
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[r] = mfma_coded(join(w[r][0], w[r][1]), join(x[0], x[1]), acc[r], sw, sx);
  }
  __shared__ float part[NW][16][16];  // [wave][token][row], a row tile at a time
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    __syncthreads();
    *reinterpret_cast<f32x4 *>(&part[wave][r16][g * 4]) = acc[r];
    __syncthreads();
    if (threadIdx.x < 256) {
      const int t = threadIdx.x >> 4, q = threadIdx.x & 15, n = n0 + r * 16 + q;
      if (t < a.T && n < a.N) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < NW; ++i) s += part[i][t][q];
        if (a.P)
          a.P[(static_cast<int64_t>(sl) * a.T + t) * a.ldp + n] = s;
        else
          a.Y[static_cast<int64_t>(t) * a.N + n] = f32_to_bf16(s);
      }
    }
  }
}

// ---- many tokens: LDS-tiled product --------------------------------------------
// A workgroup owns BM weight rows (A operand) x BN tokens.  A stage is one
// 128-k block: 128 bytes of every row, 16-byte chunk c of row r in slot c ^
// (r / 2 % 8) -- the 16 lanes of a read phase hold 16 rows of a 32-row fragment
// and one chunk, and that spreads them over all 64 banks (c ^ (r % 8), which
// suits 16-row fragments, met in half of them) -- and behind the rows each wave's copy of the
// block's scale bytes of its tokens; the weights' one scale byte per wave and
// block comes from a register that holds the next 64 blocks', one per lane.
// The waves work in 64-deep halves of it with the 32 x 32 x 64 instruction,
// whose fragments are half a stage deep: while one half is multiplied from
// registers the next is read from LDS and further stages are in flight.  (The
// 16 x 16 x 128 instruction needs all of a stage's fragments at once: with
// loads, reads and MFMAs in turn a 2048 x 21504 x 5376 call took 231 us.)
typedef float f32x16 __attribute__((ext_vector_type(16)));

// D += 2^(sa-127) 2^(sb-127) A B for a 32 x 32 tile over 64 k: lane l supplies
// 32 codes of A row l & 31 and of B column l & 31 and the scale byte of each;
// element i of D is row 8 (i / 4) + 4 (l >> 5) + i % 4, column l & 31.
__device__ __forceinline__ f32x16 mfma_coded32(i32x8 a, i32x8 b, f32x16 c, int sa, int sb) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 0, sa, 0, sb);
}

template <int BM_, int BN_, int WM_, int WN_, int NST_>
struct CTile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NST = NST_;
  static constexpr int NW = WM * WN;
  static constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 32, FN = TN / 32;
  static constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW, LPW = LA + LB + 1;  // load instructions of a wave per stage
  static constexpr int BOFF = BM * kRowBytes, SCALES = BOFF + BN * kRowBytes;  // 256 scale bytes per wave
  static constexpr int STAGE = SCALES + NW * 256;
  static constexpr int PITCH = 2 * BM + 16;  // staged output tile: bytes per token row
  static constexpr size_t RING = static_cast<size_t>(NST) * STAGE, OUT = static_cast<size_t>(BN) * PITCH;
  static constexpr size_t LDS = RING > OUT ? RING : OUT;
  static_assert(BM / 8 % NW == 0 && BN / 8 % NW == 0 && kBlk % TM == 0 && BN <= 256 && NW >= 2, "tile shape");
  static_assert(LDS <= 160 * 1024, "ring");
};

template <typename TL>
__global__ __launch_bounds__(TL::NW * 64) __attribute__((amdgpu_waves_per_eu(1, TL::LDS > 80 * 1024 ? 2 : 4))) void
coded_gemm_kernel(CodedArgs a) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / TL::WN, wn = wave % TL::WN;
  const int r32 = lane & 31, g = lane >> 5;
  int f, sl, t;
  unit_of(blockIdx.x, a.nM * a.nT * a.ksplit, a.nT, a.ksplit, f, sl, t);
  const int m0 = f * TL::BM, n0 = t * TL::BN;
  const int s0 = min(a.nb, sl * a.steps_per_slice), nk = min(a.nb, s0 + a.steps_per_slice) - s0;

  // One descriptor per operand, based at the tile's first row and this slice's
  // first k; a load instruction covers 8 rows, its first by the scalar offset.
  const auto rw = tile_rsrc(a.W + static_cast<int64_t>(m0) * a.K + static_cast<int64_t>(s0) * kBlk);
  const auto rx = tile_rsrc(a.X + static_cast<int64_t>(n0) * a.K + static_cast<int64_t>(s0) * kBlk);
  const int lrow = lane >> 3;
  const uint32_t lo = static_cast<uint32_t>(lrow) * a.K + ((lane & 7) ^ (lrow >> 1)) * 16;
  const int limw = a.N - m0, limx = a.T - n0, K8 = __builtin_amdgcn_readfirstlane(8 * a.K);
  // This wave's token scales of a block: a dword of four tokens per lane.
  const int tok0 = n0 + wn * TL::TN;
  const auto rs = tile_rsrc(a.sx + static_cast<int64_t>(s0) * a.ldsx);
  const uint32_t slo = lane * 4 < TL::TN && tok0 + lane * 4 < a.ldsx ? tok0 + lane * 4 : kBufNoRow;
  const uint8_t *swp = a.sw + static_cast<int64_t>(s0) * a.ldsw + (m0 + wm * TL::TM) / kBlk;
  auto weight_scales = [&](int kt) { return static_cast<int>(swp[static_cast<int64_t>(min(kt + lane, nk - 1)) * a.ldsw]); };
  // Stage loads past the last block read no rows (zeros), so that the loop
  // needs no branches and counts the same loads in flight at every step.
  int issued = 0;
  auto issue = [&](int stage) __attribute__((always_inline)) {
    const bool live = issued < nk;
    uint8_t *st = lds + stage;
#pragma unroll
    for (int q = 0; q < TL::LA; ++q) {
      const int gq = wave * TL::LA + q;
      load_lds<16>(rw, live && gq * 8 + lrow < limw ? lo ^ (64 * (gq & 1)) : kBufNoRow, st + gq * 1024, gq * K8 + issued * kBlk);
    }
#pragma unroll
    for (int q = 0; q < TL::LB; ++q) {
      const int gq = wave * TL::LB + q;
      load_lds<16>(rx, live && gq * 8 + lrow < limx ? lo ^ (64 * (gq & 1)) : kBufNoRow, st + TL::BOFF + gq * 1024, gq * K8 + issued * kBlk);
    }
    load_lds<4>(rs, live ? slo : kBufNoRow, st + TL::SCALES + wave * 256, live ? issued * a.ldsx : 0);
    ++issued;
  };

  f32x16 acc[TL::FM][TL::FN];
#pragma unroll
  for (int i = 0; i < TL::FM; ++i)
#pragma unroll
    for (int j = 0; j < TL::FN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
  // fragment reads: chunks 4 h + 2 g and + 1 of the row
  const int arow = (wm * TL::TM + r32) * kRowBytes, brow = TL::BOFF + (wn * TL::TN + r32) * kRowBytes;
  const int c0 = ((2 * g) ^ ((r32 >> 1) & 7)) * 16, c1 = ((2 * g + 1) ^ ((r32 >> 1) & 7)) * 16;
  const int sxoff = TL::SCALES + wave * 256 + r32;
  auto read = [&](i32x8(&fa)[TL::FM], i32x8(&fb)[TL::FN], int stage, int h) __attribute__((always_inline)) {
    const uint8_t *sb = lds + stage;
#pragma unroll
    for (int j = 0; j < TL::FN; ++j)
      fb[j] = join(*reinterpret_cast<const u32x4 *>(sb + brow + j * 32 * kRowBytes + (c0 ^ (64 * h))),
                   *reinterpret_cast<const u32x4 *>(sb + brow + j * 32 * kRowBytes + (c1 ^ (64 * h))));
#pragma unroll
    for (int i = 0; i < TL::FM; ++i)
      fa[i] = join(*reinterpret_cast<const u32x4 *>(sb + arow + i * 32 * kRowBytes + (c0 ^ (64 * h))),
                   *reinterpret_cast<const u32x4 *>(sb + arow + i * 32 * kRowBytes + (c1 ^ (64 * h))));
  };
  int sx[TL::FN], nx[TL::FN], sw = 0;
  auto read_scales = [&](int(&x)[TL::FN], int stage) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < TL::FN; ++j) x[j] = lds[stage + sxoff + j * 32];
  };
  auto multiply = [&](const i32x8(&fa)[TL::FM], const i32x8(&fb)[TL::FN]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < TL::FM; ++i)
#pragma unroll
      for (int j = 0; j < TL::FN; ++j) acc[i][j] = mfma_coded32(fa[i], fb[j], acc[i][j], sw, sx[j]);
  };

  i32x8 a0[TL::FM], b0[TL::FN], a1[TL::FM], b1[TL::FN];
#pragma unroll
  for (int st = 0; st < TL::NST; ++st) issue(st * TL::STAGE);
  wait_and_sync<(TL::NST - 1) * TL::LPW>();
  int cur = 0;
  read(a0, b0, 0, 0);
  read_scales(sx, 0);
  constexpr int kMfma = TL::FM * TL::FN, kReads = 2 * (TL::FM + TL::FN);
  for (int base = 0; base < nk; base += 64) {
    const int wv = weight_scales(base), n = min(64, nk - base);
    for (int kt = 0; kt < n; ++kt) {
      sw = __builtin_amdgcn_readlane(wv, kt);
      read(a1, b1, cur, 1);
      multiply(a0, b0);
      lead_mfma<kMfma, kReads, 0>();
      // every wave has read all of this stage: its buffer takes the loads of
      // the stage NST ahead; the next stage has landed
      wait_and_sync<(TL::NST - 2) * TL::LPW>();
      issue(cur);
      cur = cur + TL::STAGE == static_cast<int>(TL::RING) ? 0 : cur + TL::STAGE;
      read_scales(nx, cur);
      read(a0, b0, cur, 0);
      multiply(a1, b1);
      lead_mfma<kMfma, kReads + TL::FN, TL::LPW>();
#pragma unroll
      for (int j = 0; j < TL::FN; ++j) sx[j] = nx[j];
    }
  }
  wait_and_sync<0>();  // the ring is idle

  if (a.P) {
    float *P = a.P + static_cast<int64_t>(sl) * a.T * a.ldp;
#pragma unroll
    for (int j = 0; j < TL::FN; ++j) {
      const int tok = n0 + wn * TL::TN + j * 32 + r32;
      if (tok >= a.T) continue;
#pragma unroll
      for (int i = 0; i < TL::FM; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int row = m0 + wm * TL::TM + i * 32 + q * 8 + g * 4;
          if (row < a.ldp)
            *reinterpret_cast<f32x4 *>(P + static_cast<int64_t>(tok) * a.ldp + row) =
                f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        }
    }
    return;
  }
  // token-major bf16 tile in LDS, then whole 16-byte chunks of y rows
#pragma unroll
  for (int j = 0; j < TL::FN; ++j)
#pragma unroll
    for (int i = 0; i < TL::FM; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int tl = wn * TL::TN + j * 32 + r32, fl = wm * TL::TM + i * 32 + q * 8 + g * 4;
        *reinterpret_cast<uint2 *>(lds + tl * TL::PITCH + fl * 2) = make_uint2(
            pack_bf16(acc[i][j][4 * q], acc[i][j][4 * q + 1]),
            pack_bf16(acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]));
      }
  __syncthreads();
  constexpr int CPR = TL::BM / 8;
  for (int c = threadIdx.x; c < TL::BN * CPR; c += TL::NW * 64) {
    const int tl = c / CPR, fl = (c % CPR) * 8;
    const int tok = n0 + tl, row = m0 + fl;
    if (tok >= a.T || row >= a.N) continue;
    const uint4 v = *reinterpret_cast<const uint4 *>(lds + tl * TL::PITCH + fl * 2);
    uint16_t *p = a.Y + static_cast<int64_t>(tok) * a.N + row;
    if (row + 8 <= a.N && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
      *reinterpret_cast<uint4 *>(p) = v;
    } else {
      const uint32_t o[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (row + e < a.N) p[e] = static_cast<uint16_t>(o[e / 2] >> (16 * (e & 1)));
    }
  }
}

// y = bf16(sum of the K slices, in slice order), four rows per thread.
__global__ __launch_bounds__(256) void coded_sum_kernel(const float *P, int ksplit, int T, int N, int ldp, uint16_t *Y) {
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int q = ldp / 4;
  if (id >= static_cast<int64_t>(T) * q) return;
  const int64_t tok = id / q;
  const int row = static_cast<int>(id % q) * 4;
  f32x4 s{0.f, 0.f, 0.f, 0.f};
  for (int i = 0; i < ksplit; ++i)
    s += *reinterpret_cast<const f32x4 *>(P + (static_cast<int64_t>(i) * T + tok) * ldp + row);
  uint16_t *p = Y + tok * N + row;
  if (row + 4 <= N && (reinterpret_cast<uintptr_t>(p) & 7) == 0) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16(s[0], s[1]),
                                               pack_bf16(s[2], s[3]));
  } else {
    for (int e = 0; e < 4 && row + e < N; ++e) p[e] = f32_to_bf16(s[e]);
  }
}

struct CPlan {
  int tile, ksplit, per, nM, nT;
};

// Tile shapes with the us of one k step of a workgroup alone on its CU (fitted
// at K = 5376 and 21504); 128 x 128 workgroups also run two to a CU, on a ring
// of two stages, when there are more of them than CUs.
struct CShape {
  int BM, BN;
  double step;
};
constexpr CShape kShapes[] = {{256, 256, 1.62}, {256, 128, 1.03}, {128, 128, 0.8}, {128, 64, 0.58}};
constexpr int kShape128 = 2;
constexpr double kPairStep = 1.15;

// Tile shape and K split of the product: the smallest estimated time, rounds
// of workgroups over the CUs times the steps of one (3 more for its start and
// end), plus writing and summing the partials when K is split.  (21504 x 5376,
// us by shape: T = 256 58, 49, 57, 68; T = 512 73, 88, 96, 125; 8192 x 5376 at T =
// 1024 54, 43, 47, 79; 4096 x 1152 at T = 256 15, 11, 8, 7.)
CPlan plan_coded(int N, int T, int nb) {
  CPlan best{};
  double best_us = 1e300;
  for (int i = 0; i < 4; ++i) {
    const CShape &sh = kShapes[i];
    const int nM = (N + sh.BM - 1) / sh.BM, nT = (T + sh.BN - 1) / sh.BN;
    const int64_t tiles = static_cast<int64_t>(nM) * nT;
    for (int ks = 1; ks <= 16 && ks * 2 <= std::max(2, nb); ++ks) {
      const int per = (nb + ks - 1) / ks;
      if ((ks - 1) * per >= nb) continue;  // an empty slice
      const bool pairs = i == kShape128 && tiles * ks > kCUs;
      const int64_t slots = pairs ? 2 * kCUs : kCUs;
      const double rounds = static_cast<double>((tiles * ks + slots - 1) / slots);
      double us = rounds * (per + 3) * (pairs ? kPairStep : sh.step);
      if (ks > 1) us += 4.0 + 2.0 * ks * static_cast<double>(T) * N * 4 / 3e6;
      if (us < best_us) {
        best_us = us;
        best = CPlan{i, ks, per, nM, nT};
      }
    }
  }
  return best;
}

// Slices of the several-token stream, 0 for the one-tile kernel (which needs
// none).  It pays for its summing launch (4 us) where the x loads it saves are
// worth more: from 64 M codes on (several weights in turn, 21504 x 5376 at T =
// 16: 30.6 us against 33.3, 5376 x 21504: 28.8 against 39.5; 8192 x 5376: 13.2
// against 12.2, 4096 x 5376: 10.4 against 7.3).  The slices are the fewest whose workgroups come
// within 15% of whole rounds of the CUs, of at least 8 blocks (one per wave).
int wide_slices(int N, int T, int nb) {
  if (T <= kNarrowT || static_cast<int64_t>(N) * nb * kBlk < (int64_t{64} << 20)) return 0;
  const int tiles = (N + kWideRows - 1) / kWideRows;
  const int least = (nb + kStreamSlice - 1) / kStreamSlice;
  int best = 0;
  double best_eff = 0.0;
  for (int ks = least; ks <= std::max(least, 12); ++ks) {
    const int per = (nb + ks - 1) / ks;
    if (per < 8 && ks > least) break;
    if ((ks - 1) * per >= nb) continue;  // an empty slice
    const int units = tiles * ks, rounds = (units + kCUs - 1) / kCUs;
    const double eff = static_cast<double>(units) / (rounds * kCUs);
    if (units < 3 * kCUs / 4) continue;
    if (eff > best_eff) {
      best_eff = eff;
      best = ks;
    }
    if (eff >= 0.85) break;
  }
  return best;
}

template <typename TL>
hipError_t launch_coded_tile(const CodedArgs &a, hipStream_t stream) {
  const hipError_t e = ensure_lds<coded_gemm_kernel<TL>>(TL::LDS);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(coded_gemm_kernel<TL>, dim3(a.nM * a.nT * a.ksplit), dim3(TL::NW * 64), TL::LDS, stream, a);
  return hipGetLastError();
}

}  // namespace

size_t coded_partial_bytes(int N, int T, int K) {
  const int nb = (K + kBlk - 1) / kBlk;
  const int ks = T <= kDecodeMaxT ? wide_slices(N, T, nb) : plan_coded(N, T, nb).ksplit;
  return ks > 1 ? static_cast<size_t>(ks) * T * ((N + 3) & ~3) * 4 : 0;
}

hipError_t launch_encode_act(const uint16_t *x, int T, int K, const CodedView &o, hipStream_t stream) {
  const dim3 grid((T + 15) / 16, (o.nb + kEncBlocks - 1) / kEncBlocks);
  hipLaunchKernelGGL(encode_act_kernel, grid, dim3(256), 0, stream, x, T, K, o.nb, const_cast<uint8_t *>(o.codes),
                     const_cast<uint8_t *>(o.scales), o.ldsc);
  return hipGetLastError();
}

hipError_t launch_encode_weight(const uint16_t *w, int N, int K, const CodedView &o, hipStream_t stream) {
  const dim3 grid(o.nb, (N + kBlk - 1) / kBlk);
  hipLaunchKernelGGL(encode_weight_kernel, grid, dim3(256), 0, stream, w, N, K, o.nb, const_cast<uint8_t *>(o.codes),
                     const_cast<uint8_t *>(o.scales), o.ldsc);
  return hipGetLastError();
}

hipError_t launch_expand_act(const CodedView &c, int T, uint16_t *x, int K, hipStream_t stream) {
  const dim3 grid(T, (c.nb * (kBlk / 8) + 255) / 256);
  hipLaunchKernelGGL(expand_act_kernel, grid, dim3(256), 0, stream, c, x, K);
  return hipGetLastError();
}

namespace {

// y = bf16 of the sum of the slices' partials
hipError_t launch_coded_sum(const CodedArgs &a, hipStream_t stream) {
  const int64_t n = static_cast<int64_t>(a.T) * (a.ldp / 4);
  hipLaunchKernelGGL(coded_sum_kernel, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0, stream,
                     static_cast<const float *>(a.P), a.ksplit, a.T, a.N, a.ldp, a.Y);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_coded_linear(const CodedView &w, int N, const uint16_t *src, int K, const CodedView &x, int T,
                               uint16_t *y, float *partials, hipStream_t stream) {
  CodedArgs a{};
  a.W = w.codes;
  a.sw = w.scales;
  a.ldsw = w.ldsc;
  a.X = x.codes;
  a.sx = x.scales;
  a.ldsx = x.ldsc;
  a.Y = y;
  a.N = N;
  a.T = T;
  a.nb = w.nb;
  a.K = w.nb * kBlk;
  a.ldp = (N + 3) & ~3;
  hipError_t e;
  const bool fuse = src && T <= kFuseT;
  if (src && !fuse) {
    e = launch_encode_act(src, T, K, x, stream);
    if (e != hipSuccess) return e;
  }
  if (T <= kDecodeMaxT) {
    a.ksplit = wide_slices(N, T, a.nb);
    if (a.ksplit) {
      a.steps_per_slice = (a.nb + a.ksplit - 1) / a.ksplit;
      a.P = a.ksplit > 1 ? partials : nullptr;
      const int tiles = (N + kWideRows - 1) / kWideRows;
      hipLaunchKernelGGL(coded_wide_kernel, dim3(tiles * a.ksplit), dim3(kWideWaves * 64), 0, stream, a);
      e = hipGetLastError();
      return e != hipSuccess || a.ksplit == 1 ? e : launch_coded_sum(a, stream);
    }
    const int rounds = (N + 16 * kCUs - 1) / (16 * kCUs);
    a.rows = (N + rounds * kCUs - 1) / (rounds * kCUs);
    const dim3 grid((N + a.rows - 1) / a.rows);
    if (fuse) {
      a.x = src;
      a.Kx = K;
      hipLaunchKernelGGL(coded_stream_kernel<true>, grid, dim3(kStreamWaves * 64), 0, stream, a);
    } else {
      hipLaunchKernelGGL(coded_stream_kernel<false>, grid, dim3(kStreamWaves * 64), 0, stream, a);
    }
    return hipGetLastError();
  }
  const CPlan p = plan_coded(N, T, a.nb);
  a.nM = p.nM;
  a.nT = p.nT;
  a.ksplit = p.ksplit;
  a.steps_per_slice = p.per;
  a.P = p.ksplit > 1 ? partials : nullptr;
  switch (p.tile) {
    case 0: e = launch_coded_tile<CTile<256, 256, 2, 4, 2>>(a, stream); break;
    case 1: e = launch_coded_tile<CTile<256, 128, 4, 2, 3>>(a, stream); break;
    case kShape128:
      e = p.nM * p.nT * p.ksplit > kCUs ? launch_coded_tile<CTile<128, 128, 2, 4, 2>>(a, stream)
                                        : launch_coded_tile<CTile<128, 128, 2, 4, 4>>(a, stream);
      break;
    default: e = launch_coded_tile<CTile<128, 64, 4, 2, 4>>(a, stream); break;
  }
  return e != hipSuccess || p.ksplit == 1 ? e : launch_coded_sum(a, stream);
}

}  // namespace wl
