// Device coding of and access to 8-bit blocks (coded.hip describes the coding), and
// the conversion to bf16 that goes with it.
#pragma once

#include "common.h"
#include "training.h"

namespace wl {

constexpr int kCodeBlock = 128;

// Two floats -> two bf16 in one instruction (nearest-even, NaN stays NaN); a in
// the low half.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}

// Elements k .. k + 7 (k % 8 == 0) of row t: code * 2^e as bf16, exact.
__device__ __forceinline__ u32x4 expand8(const CodedView &c, int64_t t, int k) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const u32x2 v = *reinterpret_cast<const u32x2 *>(c.codes + t * (c.nb * kCodeBlock) + k);
  const float f = __uint_as_float(static_cast<uint32_t>(c.scales[static_cast<int64_t>(k / kCodeBlock) * c.ldsc + t]) << 23);
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

}  // namespace wl
