// Device access to 8-bit coded activations (coded.hip describes the coding), and
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

}  // namespace wl
