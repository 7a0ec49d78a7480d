// Root-mean-square norm with the residual's addition and a coded output, and
// its backward pass.
//
// Forward, for each token row:
//   h = bf16(x + res)            (h = x without a residual)
//   a = 1 / sqrt(mean_k h_k^2 + eps)
//   y = bf16(h a (offset + w))   code = the 8-bit coding of y (coded.h)
// Backward, with g = dy (offset + w) and n = h a:
//   dx = a (g - n mean_k(g n)) + dh      dw = sum_t dy n
//
// Both are bound by memory: a row is read once into registers, 16 bytes a lane
// and load, and everything that follows comes from there.  One to sixteen
// waves share a row (rows of up to 32768 elements); a coded block of 128 is 16
// neighbouring lanes, so its maximum is four lane exchanges and the bf16 output
// is coded without being read again.
// Measured: 8192 x 5376 with residual, h, y and code 79 us (5.0 TB/s), or 70
// where the outputs' memory was written by the call before; its backward pass 60 (5.9
// TB/s) and 5.5 for the sum of dw; 1 x 1152 2.9 us, a launch; the backward pass of
// 333 x 1160 4.0.
#include <algorithm>
#include <type_traits>

#include "beside.h"
#include "coded.h"
#include "common.h"
#include "lds_dma.h"
#include "streams.h"

namespace wl {

namespace {

constexpr int kRowsOneWave = 4;  // rows of a workgroup where a wave takes a row

__device__ __forceinline__ float lo_f32(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_f32(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// ONCE: past the caches (kLastCache).
template <bool ONCE>
__device__ __forceinline__ u32x4 ld_row(const uint16_t *p) {
  return ONCE ? ld16_once(p) : ld16(p);
}

// 8 elements of the weight from k on, plus `offset`.
template <bool F32>
__device__ __forceinline__ void load_weight(const NormWeight &nw, int k, float (&w)[8], float offset) {
  if constexpr (F32) {
    const float *p = static_cast<const float *>(nw.w) + k;
    const f32x4 a = *reinterpret_cast<const f32x4 *>(p), b = *reinterpret_cast<const f32x4 *>(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = offset + a[i];
      w[4 + i] = offset + b[i];
    }
  } else {
    const u32x4 v = ld16(static_cast<const uint16_t *>(nw.w) + k);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[2 * i] = offset + lo_f32(v[i]);
      w[2 * i + 1] = offset + hi_f32(v[i]);
    }
  }
}

// Sum over the lanes of a wave, then over the W waves of a row, in a fixed order.
template <int W, typename F>
__device__ __forceinline__ F row_sum(F v, F *lds, int wave) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d, 64);
  if constexpr (W > 1) {
    if ((threadIdx.x & 63) == 0) lds[wave] = v;
    __syncthreads();
    v = lds[0];
#pragma unroll
    for (int i = 1; i < W; ++i) v += lds[i];
  }
  return v;
}

// Two doubles to bf16 with one rounding: first to float32, an inexact one towards the
// neighbour whose last bit is odd, which is never halfway between two bf16.
__device__ __forceinline__ uint32_t pack_bf16_once(double a, double b) {
  const auto odd = [](double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = static_cast<uint32_t>(u), cut = lo & 0xe0000000u;
    const uint64_t o = (u & 0xffffffff00000000u) | (lo != cut ? cut | 0x20000000u : cut);
    return static_cast<float>(__builtin_bit_cast(double, o));
  };
  return pack_bf16(odd(a), odd(b));
}

// y of 8 elements h of a row: h a (offset + w), rounded once, so that y and its codes are
// those of exact arithmetic.
__device__ __forceinline__ u32x4 scale_row(u32x4 h, double a, const float (&w)[8], double offset) {
  u32x4 y;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t v = h[j];
    asm("" : "+v"(v));  // (converted again here: kept from the sum of squares they take twice the registers)
    y[j] = pack_bf16_once(lo_f32(v) * a * (offset + w[2 * j]), hi_f32(v) * a * (offset + w[2 * j + 1]));
  }
  return y;
}

// W waves to a row (1: kRowsOneWave rows to a workgroup), V vectors of 8 a lane.
// The sum of squares, a and the product are taken in 64 bits: about a dozen such
// operations an element.  (With the product in float32, rounded a second time, 12 to 26 of
// the 44 million codes of 8192 x 5376 were others, and 65.6 us instead of 70; only the
// vectors next to a halfway value in 64 bits: 69.5.)
template <int W, int V, bool F32, bool ONCE>
__global__ __launch_bounds__(W == 1 ? kRowsOneWave * 64 : W * 64) void norm_kernel(NormCall c) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = W == 1 ? static_cast<int64_t>(blockIdx.x) * kRowsOneWave + wave : blockIdx.x;
  if (W == 1 && t >= c.T) return;  // (no barrier in that form)
  const int at = (W == 1 ? lane : static_cast<int>(threadIdx.x)) * 8;
  __shared__ double part[W];
  const int64_t row = t * c.K;
  u32x4 h[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int k = at + i * W * 512;
    h[i] = u32x4{0u, 0u, 0u, 0u};
    if (k < c.K) h[i] = ld_row<ONCE>(c.x + row + k);
  }
  float w[8];  // (one vector a lane: under way with the row)
  if (V == 1 && at < c.K) load_weight<F32>(c.w, at, w, 0.f);
  if (c.res) {
    u32x4 r[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int k = at + i * W * 512;
      r[i] = u32x4{0u, 0u, 0u, 0u};
      if (k < c.K) r[i] = ld_row<ONCE>(c.res + row + k);
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        h[i][j] = pack_bf16(lo_f32(h[i][j]) + lo_f32(r[i][j]), hi_f32(h[i][j]) + hi_f32(r[i][j]));
  }
  if (c.h) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int k = at + i * W * 512;
      if (k < c.K) *reinterpret_cast<u32x4 *>(c.h + row + k) = h[i];
    }
  }
  double q = 0.0;
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const double a = lo_f32(h[i][j]), b = hi_f32(h[i][j]);
      q = __builtin_fma(a, a, q);
      q = __builtin_fma(b, b, q);
    }
  q = row_sum<W>(q, part, wave);
  const double a = rsqrt(q / c.K + static_cast<double>(c.eps));
  if (c.rstd && at == 0) c.rstd[t] = static_cast<float>(a);
  if (!c.y && !c.coded) return;
  const int Kq = c.code.nb * kCodeBlock;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int k = at + i * W * 512;
    u32x4 y{0u, 0u, 0u, 0u};
    if (k < c.K) {
      if (V > 1) load_weight<F32>(c.w, k, w, 0.f);
      y = scale_row(h[i], a, w, c.w.offset);
      if (c.y) *reinterpret_cast<u32x4 *>(c.y + row + k) = y;
    }
    if (c.coded) {
      uint32_t m = amax_bits(y);
#pragma unroll
      for (int d = 1; d < 16; d <<= 1) m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), d, 16)));
      const int e = block_exponent(m), l = lane & 15;
      if (k < Kq) {
        *reinterpret_cast<u32x2 *>(const_cast<uint8_t *>(c.code.codes) + t * Kq + k) = code8(y, e);
        uint8_t *s = const_cast<uint8_t *>(c.code.scales) + static_cast<int64_t>(k / kCodeBlock) * c.code.ldsc + t;
        if (l == 0) *s = static_cast<uint8_t>(e + 127);
        // behind the last token the run of a block is filled up with scale 1
        else if (t == c.T - 1 && t + l < c.code.ldsc) s[l] = 127;
      }
    }
  }
}

__device__ __forceinline__ void load_8(const float *p, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const f32x4 x = reinterpret_cast<const f32x4 *>(p)[j];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[4 * j + i] = x[i];
  }
}
__device__ __forceinline__ void store_8(float *p, const float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 2; ++j) reinterpret_cast<f32x4 *>(p)[j] = f32x4{v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]};
}

template <int W, int V>
constexpr bool in_lds() { return W == 16 && V > 2; }

// dw of 64 columns from all rows, which the waves take in turn, 8 at a time.
template <int WAVES>
__device__ __forceinline__ void dw_columns(const NormBackward &c, int unit) {
  constexpr int AHEAD = 4;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = unit * 64 + (lane & 7) * 8;
  const bool in = col < c.K;
  float dw[8] = {};
  for (int t0 = wave * 8 + (lane >> 3); t0 < c.T; t0 += 8 * WAVES * AHEAD) {
    u32x4 d[AHEAD], h[AHEAD];
    float a[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int64_t t = min(t0 + 8 * WAVES * i, c.T - 1), at = t * c.K + (in ? col : 0);
      d[i] = ld16(c.dy + at);
      h[i] = ld16(c.h + at);
      a[i] = c.rstd[t];
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const bool row = t0 + 8 * WAVES * i < c.T;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n = (j & 1 ? hi_f32(h[i][j / 2]) : lo_f32(h[i][j / 2])) * a[i];
        const float g = j & 1 ? hi_f32(d[i][j / 2]) : lo_f32(d[i][j / 2]);
        dw[j] = row ? __builtin_fmaf(g, n, dw[j]) : dw[j];
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int x = 8; x < 64; x <<= 1) dw[j] += __shfl_xor(dw[j], x, 64);
  __shared__ float part[WAVES][64];
  if (lane < 8) store_8(&part[wave][lane * 8], dw);
  __syncthreads();
  const int k = unit * 64 + static_cast<int>(threadIdx.x);
  if (threadIdx.x < 64 && k < c.K) {
    float s = part[0][threadIdx.x];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) s += part[w][threadIdx.x];
    c.dw[k] = s;
  }
}

// Backward.  A team of W waves walks the rows `team`, `team` + teams, ...; its
// sum of dy n stays with it, the workgroup's sums (a row of K floats) go to
// `part` (dw itself if there is one workgroup).  With few rows dw has workgroups of
// its own, 64 columns each, behind the `groups` of the rows: they read the rows again,
// from the caches, and no second launch is needed.
template <int W, int V, bool F32, bool ONCE>
__global__ __launch_bounds__(W == 1 ? kRowsOneWave * 64 : W * 64) void norm_backward_kernel(NormBackward c, float *part, int groups) {
  if (static_cast<int>(blockIdx.x) >= groups) return dw_columns<W == 1 ? kRowsOneWave : W>(c, blockIdx.x - groups);
  constexpr int R = W == 1 ? kRowsOneWave : 1;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int at = (W == 1 ? lane : static_cast<int>(threadIdx.x)) * 8;
  __shared__ float sum[2][W];
  // the weight stays in registers but for sixteen waves of several vectors, which read
  // it again for each row (kept, it spills)
  constexpr bool KEPT = W < 16 || V == 1;
  // and dw but for the longest rows, each lane's in LDS (2048 rows of 21504: 136 us with
  // dw in registers, which spill, so 79)
  constexpr bool IN_LDS = in_lds<W, V>();
  extern __shared__ __align__(16) float sums[];  // [K]
  float w[KEPT ? V : 1][8], dw[IN_LDS ? 1 : V][8];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int k = at + i * W * 512;
#pragma unroll
    for (int j = 0; j < 8; ++j) w[KEPT ? i : 0][j] = dw[IN_LDS ? 0 : i][j] = 0.f;
    if (KEPT && k < c.K) load_weight<F32>(c.w, k, w[KEPT ? i : 0], c.w.offset);
    if (IN_LDS && k < c.K) store_8(sums + k, dw[0]);
  }
  const int64_t teams = static_cast<int64_t>(groups) * R;
  int turn = 0;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * R + (W == 1 ? wave : 0); t < c.T; t += teams, turn ^= 1) {
    const int64_t row = t * c.K;
    u32x4 d[V], h[V], r[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int k = at + i * W * 512;
      d[i] = h[i] = r[i] = u32x4{0u, 0u, 0u, 0u};
      if (k < c.K) {
        d[i] = ld_row<ONCE>(c.dy + row + k);
        h[i] = ld_row<ONCE>(c.h + row + k);
        if (c.dh && !IN_LDS) r[i] = ld_row<ONCE>(c.dh + row + k);
      }
    }
    const float a = c.rstd[t];
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int k = at + i * W * 512;
      float(&wi)[8] = w[KEPT ? i : 0];
      if (!KEPT && k < c.K) load_weight<F32>(c.w, k, wi, c.w.offset);
      float(&dwi)[8] = dw[IN_LDS ? 0 : i];
      if (IN_LDS && k < c.K) load_8(sums + k, dwi);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n = (j & 1 ? hi_f32(h[i][j / 2]) : lo_f32(h[i][j / 2])) * a;
        const float g = j & 1 ? hi_f32(d[i][j / 2]) : lo_f32(d[i][j / 2]);
        // (past the row g is 0 and w of the vector before it may not be finite)
        dot = KEPT || k < c.K ? __builtin_fmaf(g * wi[j], n, dot) : dot;
        dwi[j] = __builtin_fmaf(g, n, dwi[j]);
      }
      if (IN_LDS && k < c.K) store_8(sums + k, dwi);
    }
    if (!c.dx) continue;
    const float mean = row_sum<W>(dot, sum[turn], wave) / c.K;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int k = at + i * W * 512;
      if (k >= c.K) continue;
      float(&wi)[8] = w[KEPT ? i : 0];
      if (!KEPT) load_weight<F32>(c.w, k, wi, c.w.offset);
      if (c.dh && IN_LDS) r[i] = ld_row<ONCE>(c.dh + row + k);
      u32x4 o;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float n0 = lo_f32(h[i][j]) * a, n1 = hi_f32(h[i][j]) * a;
        const float g0 = lo_f32(d[i][j]) * wi[2 * j], g1 = hi_f32(d[i][j]) * wi[2 * j + 1];
        o[j] = pack_bf16(__builtin_fmaf(a, __builtin_fmaf(-n0, mean, g0), lo_f32(r[i][j])),
                         __builtin_fmaf(a, __builtin_fmaf(-n1, mean, g1), hi_f32(r[i][j])));
      }
      *reinterpret_cast<u32x4 *>(c.dx + row + k) = o;
    }
  }
  if (!c.dw || gridDim.x > static_cast<uint32_t>(groups)) return;
  float *out = (groups == 1 ? c.dw : part) + static_cast<int64_t>(blockIdx.x) * c.K;
  if constexpr (R == 1) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int k = at + i * W * 512;
      if (k >= c.K) continue;
      if constexpr (IN_LDS) load_8(sums + k, dw[0]);
      store_8(out + k, dw[IN_LDS ? 0 : i]);
    }
  } else {
    __shared__ f32x4 rows[R - 1][64 * 2];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int k = at + i * W * 512;
      __syncthreads();
      if (wave > 0)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          rows[wave - 1][lane + 64 * j] = f32x4{dw[i][4 * j], dw[i][4 * j + 1], dw[i][4 * j + 2], dw[i][4 * j + 3]};
      __syncthreads();
      if (wave == 0 && k < c.K)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          f32x4 s = f32x4{dw[i][4 * j], dw[i][4 * j + 1], dw[i][4 * j + 2], dw[i][4 * j + 3]};
#pragma unroll
          for (int q = 0; q < R - 1; ++q) s += rows[q][lane + 64 * j];
          *reinterpret_cast<f32x4 *>(out + k + 4 * j) = s;
        }
    }
  }
}

// dw [K] = sum over G rows of part [G][K]: 16 columns a workgroup, its 16
// groups of 16 lanes take rows in turn and meet in LDS, in a fixed order.
__global__ __launch_bounds__(256) void norm_dw_kernel(const float *part, int G, int K, float *dw) {
  const int l = threadIdx.x & 15, g = threadIdx.x >> 4;
  const int k = blockIdx.x * 16 + l;
  __shared__ float s[16][17];
  float v = 0.f;
  if (k < K) {
#pragma unroll 16
    for (int i = g; i < G; i += 16) v += part[static_cast<int64_t>(i) * K + k];
  }
  s[g][l] = v;
  __syncthreads();
  if (g == 0 && k < K) {
#pragma unroll
    for (int i = 1; i < 16; ++i) v += s[i][l];
    dw[k] = v;
  }
}

__global__ __launch_bounds__(256) void fill_zero_f32(float *p, int n) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i < n) p[i] = 0.f;
}

// Waves and vectors of a row.  One vector a lane while that takes four waves or fewer
// (1 row of 2048: 5.2 -> 2.7 us, 8192 rows 30.4 -> 28.6, against one wave), and with few
// rows up to sixteen (1 row of 8192 5.6 -> 4.2, 256 rows 8.6 -> 6.9; 512 level; 2048 rows
// of 5376 20.1 -> 22.5, 8192 rows 76 -> 85); else four waves up to 8192 elements.
constexpr int kFewRows = 512;

template <typename F>
hipError_t with_row_shape(int T, int K, F &&f) {
  const auto shape = [&](auto w, auto v) { return f(w, v); };
  const std::integral_constant<int, 1> i1{};
  const std::integral_constant<int, 2> i2{};
  const std::integral_constant<int, 3> i3{};
  const std::integral_constant<int, 4> i4{};
  const std::integral_constant<int, 16> i16{};
  if (K <= 512) return shape(i1, i1);
  if (K <= 1024) return shape(i2, i1);
  if (K <= 2048) return shape(i4, i1);
  if (T <= kFewRows && K <= 4096) return shape(std::integral_constant<int, 8>{}, i1);
  if (T <= kFewRows && K <= 8192) return shape(i16, i1);
  if (K <= 4096) return shape(i4, i2);
  if (K <= 6144) return shape(i4, i3);
  if (K <= 8192) return shape(i4, i4);
  if (K <= 16384) return shape(i16, i2);
  if (K <= 24576) return shape(i16, i3);
  return shape(i16, i4);
}

int rows_of_workgroup(int K) { return K <= 512 ? kRowsOneWave : 1; }

// Workgroups of the backward pass: enough to fill the CUs, few enough that the partial
// sums stay small beside the rows (8192 rows of 5376 with 384, 512, 768, 1024: 74, 74, 82,
// 81 us in both launches; of 1536, smaller workgroups: 30, 25, 21, 22).
int backward_groups(int T, int K) {
  const int64_t groups = (static_cast<int64_t>(T) + rows_of_workgroup(K) - 1) / rows_of_workgroup(K);
  return static_cast<int>(std::min<int64_t>(groups, K <= 2048 ? 768 : K <= 16384 ? 512 : 256));
}

// dw beside dx in one launch: both launches of 16 x 5376 8.3 us, this 3.3; 333 x 1160 8.2
// and 4.0; 1024 x 1160 10.3 and 9.1, x 5376 17.9 and 14.9, x 21504 50.9 and 51.9.
constexpr int kOneLaunchRows = 1024;
bool one_backward_launch(int T, int K) { return T > rows_of_workgroup(K) && T <= kOneLaunchRows; }

// Calls that move more than the last cache holds load past it, so that it keeps what
// they write (8192 x 5376 backward 69 -> 60 us; forward 79 -> 78, and 81 -> 70 where the
// outputs' memory is used again; stores past it too: 70); the inputs of smaller calls
// often lie in it (backward of 800 x 5376, so loaded: 13 -> 15 us).
constexpr int64_t kLastCache = int64_t{256} << 20;

// f(F32, ONCE); the shapes for few rows have no ONCE.
template <int W, int V, typename F>
hipError_t with_loads(bool f32, bool once, F &&f) {
  constexpr bool kCan = W < 8 || V > 1;
  const auto with = [&](auto o) { return f32 ? f(std::true_type{}, o) : f(std::false_type{}, o); };
  if (kCan && once) return with(std::integral_constant<bool, kCan>{});
  return with(std::false_type{});
}

}  // namespace

hipError_t launch_norm(const NormCall &c, hipStream_t stream) {
  const int rows = 1 + (c.res != nullptr) + (c.h != nullptr) + (c.y != nullptr);
  const bool once = static_cast<int64_t>(c.T) * c.K * (2 * rows + c.coded) > kLastCache;
  return with_row_shape(c.T, c.K, [&](auto w, auto v) {
    constexpr int W = decltype(w)::value, V = decltype(v)::value;
    const int R = rows_of_workgroup(c.K);
    const dim3 grid((c.T + R - 1) / R), block(R * W * 64);
    return with_loads<W, V>(c.w.f32, once, [&](auto f32, auto o) {
      norm_kernel<W, V, decltype(f32)::value, decltype(o)::value><<<grid, block, 0, stream>>>(c);
      return hipGetLastError();
    });
  });
}

size_t norm_backward_partial_bytes(int T, int K) {
  const int G = backward_groups(T, K);
  return G > 1 && !one_backward_launch(T, K) ? static_cast<size_t>(G) * K * sizeof(float) : 0;
}

hipError_t launch_norm_backward(const NormBackward &c, float *partials, hipStream_t stream) {
  if (c.T == 0) {
    if (!c.dw) return hipSuccess;
    fill_zero_f32<<<(c.K + 255) / 256, 256, 0, stream>>>(c.dw, c.K);
    return hipGetLastError();
  }
  const int G = backward_groups(c.T, c.K);
  const bool one = one_backward_launch(c.T, c.K);
  if (one && c.dw && c.dx == c.dy) {  // dw has to be done with dy before dx takes its place
    NormBackward part = c;
    part.dx = nullptr;
    const hipError_t e = launch_norm_backward(part, partials, stream);
    if (e != hipSuccess) return e;
    part = c;
    part.dw = nullptr;
    return launch_norm_backward(part, partials, stream);
  }
  const bool once = static_cast<int64_t>(c.T) * c.K * 2 * (2 + (c.dh != nullptr) + (c.dx != nullptr)) > kLastCache;
  const int rows = one && !c.dx ? 0 : G, blocks = rows + (one && c.dw ? (c.K + 63) / 64 : 0);
  const hipError_t e = with_row_shape(c.T, c.K, [&](auto w, auto v) {
    constexpr int W = decltype(w)::value, V = decltype(v)::value;
    const dim3 block(rows_of_workgroup(c.K) * W * 64);
    constexpr size_t lds = in_lds<W, V>() ? sizeof(float) * W * V * 512 : 0;
    return with_loads<W, V>(c.w.f32, once, [&](auto f32, auto o) {
      constexpr auto kernel = norm_backward_kernel<W, V, decltype(f32)::value, decltype(o)::value>;
      if constexpr (lds > 0) {
        const hipError_t e = ensure_lds<kernel>(lds);
        if (e != hipSuccess) return e;
      }
      kernel<<<blocks, block, lds, stream>>>(c, partials, rows);
      return hipGetLastError();
    });
  });
  if (e != hipSuccess || !c.dw || G == 1 || one) return e;
  norm_dw_kernel<<<(c.K + 15) / 16, 256, 0, stream>>>(partials, G, c.K, c.dw);
  return hipGetLastError();
}

}  // namespace wl
