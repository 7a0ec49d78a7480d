// Pieces the staged GEMM kernels share: loads from HBM straight into LDS,
// counted waits on them, and the workgroup numbering over the XCDs.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

#include "common.h"

namespace wl {

typedef __attribute__((address_space(3))) void lds_void;

constexpr int kRowBytes = 128;  // bytes of one row per stage: 64 bf16, or 128 E4M3 codes

// LDS-DMA stage loads.  They are buffer loads into LDS (buffer_load_dwordx4
// ... lds), not global_load_lds: with the latter in flight the compiler
// drains every outstanding LDS read (s_waitcnt lgkmcnt(0)) before each use of
// a fragment, with the former it counts them (lgkmcnt(n)), so fragment reads
// stay in flight under the MFMAs (same results; the 31B prefill GEMMs ran
// 2-7% faster).  One load instruction of a wave (8 rows x 128 bytes) reads
// through one descriptor whose base is its first live lane's address less
// 128 bytes; each lane adds a 32-bit byte offset.  The rows of one
// instruction ascend with the lane (every caller maps lane >> 3 to
// consecutive rows of one operand), so every live offset is positive and
// small.  A lane without a row takes an offset past the descriptor's range,
// which the buffer unit returns as zeros.
constexpr int kBufWord3 = 0x00020000;          // raw gfx9 descriptor: no swizzle, stride 0
constexpr int kBufRange = 0x40000000;          // bytes the offsets are checked against
constexpr uint32_t kBufNoRow = 0x7ffffff0u;    // past the range: reads zeros

struct RowLoad {
  __amdgpu_buffer_rsrc_t rsrc;
  uint32_t off;  // this lane's byte offset (kBufNoRow: no row)
};

// p: this lane's source address, or null for no row; fallback: any valid
// address, the base when no lane of the wave has a row.
__device__ __forceinline__ RowLoad row_load(const void *p, const void *fallback) {
  const uint64_t live = __builtin_amdgcn_ballot_w64(p != nullptr);
  const uintptr_t addr = reinterpret_cast<uintptr_t>(p);
  uintptr_t base = reinterpret_cast<uintptr_t>(fallback);
  if (live) {
    const int first = __builtin_ctzll(live);
    const uint32_t lo = __builtin_amdgcn_readlane(static_cast<uint32_t>(addr), first);
    const uint32_t hi = __builtin_amdgcn_readlane(static_cast<uint32_t>(addr >> 32), first);
    base = ((static_cast<uintptr_t>(hi) << 32) | lo) - kRowBytes;
  }
  return RowLoad{__builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void *>(base), 0, kBufRange, kBufWord3),
                 p != nullptr ? static_cast<uint32_t>(addr - base) : kBufNoRow};
}

__device__ __forceinline__ void load_rows(const RowLoad &r, uint32_t off, uint8_t *dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r.rsrc, (lds_void *)dst, 16, off, 0, 0, 0);
}

// A descriptor at a workgroup-uniform base; lanes add byte offsets below
// kBufRange, or kBufNoRow to read zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t tile_rsrc(const void *base) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, kBufRange, kBufWord3);
}

// BYTES (4 or 16) per lane from descriptor + off (per lane) + soff (uniform) to
// dst + BYTES * lane.
template <int BYTES>
__device__ __forceinline__ void load_lds(__amdgpu_buffer_rsrc_t r, uint32_t off, uint8_t *dst, int soff) {
  static_assert(BYTES == 4 || BYTES == 16, "bytes per lane");
  if constexpr (BYTES == 16)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)dst, 16, off, soff, 0, 0);
  else
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)dst, 4, off, soff, 0, 0);
}

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | (((N >> 4) & 3) << 14));
}

// As wait_vmcnt, and every LDS read of this wave is done too; followed by the
// workgroup barrier.  The empty asm statements keep the compiler from moving
// memory operations across it.
template <int N>
__device__ __forceinline__ void wait_and_sync() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (0 << 8) | (((N >> 4) & 3) << 14));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Scheduling of a pipeline step of M MFMAs, R LDS reads and V loads into LDS:
// MFMAs first (their operands are there), the reads and loads -- for later
// steps -- spread among them, with the address arithmetic two at a time.
template <int M, int R, int V>
__device__ __forceinline__ void interleave_mfma() {
#pragma unroll
  for (int i = 0; i < M; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // one MFMA
    if ((i + 1) * V / M > i * V / M) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);  // one load
#pragma unroll
    for (int k = i * R / M; k < (i + 1) * R / M; ++k) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // one LDS read
    __builtin_amdgcn_sched_group_barrier(0x002, 2, 0);  // VALU
  }
}

// For steps of few long MFMAs: after each, an even share of the reads so that
// all are issued by three quarters of the step; the loads come first.
template <int M, int R, int V>
__device__ __forceinline__ void lead_mfma() {
  constexpr int Q = M > 1 ? (3 * M + 3) / 4 : 1;
#pragma unroll
  for (int i = 0; i < M; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if constexpr (V > 0) {
      if (i == 0) __builtin_amdgcn_sched_group_barrier(0x020, V, 0);
    }
    if (i < Q) {
#pragma unroll
      for (int k = i * R / Q; k < (i + 1) * R / Q; ++k) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
  }
}

// Workgroup index -> unit, XCD-major: hardware sends workgroup w to XCD w % 8;
// XCD x is given the contiguous unit range [x * per + min(x, rem), ...) of the
// total units.
__device__ __forceinline__ int xcd_unit(int id, int total) {
  const int x = id & 7, j = id >> 3;
  const int per = total >> 3, rem = total & 7;
  return x * per + min(x, rem) + j;
}

// Workgroup index -> (feature tile, K slice, token tile), token tile fastest.
__device__ __forceinline__ void unit_of(int id, int total, int nT, int nslices, int &f, int &sl, int &t) {
  const int u = xcd_unit(id, total);
  f = u / (nslices * nT);
  const int r = u % (nslices * nT);
  sl = r / nT;
  t = r % nT;
}

// Raise a kernel's dynamic-LDS limit to what its ring needs, once per kernel
// and device (the attribute belongs to the device the call runs on).
template <auto KERN>
inline hipError_t ensure_lds(size_t bytes) {
  static std::atomic<uint64_t> done{0};  // bit d: set on device d (d < 64)
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = dev >= 0 && dev < 64 ? (uint64_t{1} << dev) : 0;
  if (bit && (done.load(std::memory_order_acquire) & bit)) return hipSuccess;
  e = hipFuncSetAttribute(reinterpret_cast<const void *>(KERN), hipFuncAttributeMaxDynamicSharedMemorySize,
                          static_cast<int>(bytes));
  if (e == hipSuccess && bit) done.fetch_or(bit, std::memory_order_release);
  return e;
}

}  // namespace wl
