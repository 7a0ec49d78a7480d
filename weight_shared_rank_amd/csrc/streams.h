// Loads of streams that are read once.
#pragma once

#include "common.h"

namespace wl {

// 16 bytes of a stream that is read once: they leave the caches to the others.
__device__ __forceinline__ u32x4 ld16_once(const uint16_t *p) {
  return __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p));
}

}  // namespace wl
