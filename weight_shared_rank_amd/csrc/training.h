// Launches of the 8-bit coded operands (coded.hip) and of the backward pass
// (backward.hip).
#pragma once

#include "internal.h"

namespace wl {

// 8-bit coded operands (coded.hip describes the coding and the layout): codes
// [R][nb * 128] and scale bytes [nb][ldsc].
struct CodedView {
  const uint8_t *codes;
  const uint8_t *scales;
  int32_t nb;
  int32_t ldsc;
};
hipError_t launch_encode_act(const uint16_t *x, int T, int K, const CodedView &o, hipStream_t stream);
hipError_t launch_encode_weight(const uint16_t *w, int N, int K, const CodedView &o, hipStream_t stream);
// x [T][K] bf16 = code * 2^e
hipError_t launch_expand_act(const CodedView &c, int T, uint16_t *x, int K, hipStream_t stream);
// y [T][N] = x w^T; partials: coded_partial_bytes(N, T, K) bytes.  src: bf16
// [T][K] to be coded into x first, or null if x holds coded activations.
size_t coded_partial_bytes(int N, int T, int K);
hipError_t launch_coded_linear(const CodedView &w, int N, const uint16_t *src, int K, const CodedView &x, int T,
                               uint16_t *y, float *partials, hipStream_t stream);

// Backward pass of one call (backward.hip has the formulas).  c describes the
// call (x and y unused, W0 bf16), T its tokens; dy [T][columns] with the
// columns of the call's y, the tied v slot included.  Every output may be null.
struct GradOut {
  uint16_t *dx;                 // [T][K]
  float *ds;                    // [Ntot]
  uint16_t *du[kMaxChildren];   // [N][r] per child
  uint16_t *dv[kMaxChildren];   // [K][r] per child
  int32_t r[kMaxChildren];      // ranks (unpadded)
  float *dw0;                   // [Ntot][K]
  int32_t accumulate;           // dw0 is added to
};
size_t backward_workspace_bytes(const CallDesc &c, int T);
hipError_t launch_backward(const CallDesc &c, const CodedView &xc, const uint16_t *dy, const GradOut &o, void *ws,
                           hipStream_t stream);

}  // namespace wl
