// Launches of what stands before and beside a projection: the norm with the
// residual's addition and a coded output (norm.hip), and the low-rank adapters
// of many requests (adapters.hip) and their gradients (adapters_backward.hip).
#pragma once

#include "training.h"

namespace wl {

constexpr int kNormMaxK = 32768;

// The weight of a norm: bf16 or float32 [K], added to `offset`.
struct NormWeight {
  const void *w;
  bool f32;
  float offset;
};

struct NormCall {
  const uint16_t *x, *res;  // [T][K] bf16; res may be null
  int32_t T, K;
  NormWeight w;
  float eps;
  uint16_t *h, *y;          // [T][K] bf16, each may be null
  float *rstd;              // [T] or null
  bool coded;
  CodedView code;           // written if coded
};
hipError_t launch_norm(const NormCall &c, hipStream_t stream);

struct NormBackward {
  const uint16_t *dy, *h;  // [T][K] bf16
  const float *rstd;       // [T]
  const uint16_t *dh;      // [T][K] bf16 or null
  int32_t T, K;
  NormWeight w;
  uint16_t *dx;            // [T][K] bf16 or null
  float *dw;               // [K] or null
};
size_t norm_backward_partial_bytes(int T, int K);
hipError_t launch_norm_backward(const NormBackward &c, float *partials, hipStream_t stream);

// A pool of low-rank adapters beside one projection, or one stacked call.
struct AdapterPool {
  const uint16_t *vt;   // [n][nchild * r][K]
  const uint16_t *u;    // [n][Ntot][r]
  const float *scale;   // [n]
  const int32_t *rank;  // [n] or null: all r
  int32_t n, r, K, nchild;
  int32_t N[kMaxChildren];
  int32_t Ntot;
};
size_t adapters_workspace_bytes(const AdapterPool &p, int T);
// y = base + scale U (V^T x) row by row, with the adapter index[t] (none if
// outside [0, n)); y may be base.
hipError_t launch_adapters(const AdapterPool &p, const uint16_t *x, const int32_t *index, int T, const uint16_t *base,
                           uint16_t *y, void *ws, hipStream_t stream);

// Gradients of launch_adapters; every output may be null.
struct AdapterGrads {
  const uint16_t *base;  // [T][K], what dx adds to
  uint16_t *dx;          // [T][K], may be base
  uint16_t *du;          // [n][Ntot][r]
  uint16_t *dv;          // [n][nchild * r][K]
};
size_t adapters_backward_workspace_bytes(const AdapterPool &p, int T);
hipError_t launch_adapters_backward(const AdapterPool &p, const CodedView &x, const uint16_t *dy, const int32_t *index,
                                    int T, const AdapterGrads &o, void *ws, hipStream_t stream);

}  // namespace wl
