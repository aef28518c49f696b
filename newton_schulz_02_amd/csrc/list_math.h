// Device arithmetic shared by the elementwise kernels: the AdamW update of one element and the
// clip coefficient.
#pragma once

#include <hip/hip_runtime.h>

#include "list_types.h"

namespace muon {

// beta x + add, for a state x.  lo is 0 where beta is a float: its product is left out then, as
// it would make a NaN of an infinite state.
__device__ __forceinline__ float decayed(const AdamBeta& b, float x, float add) {
  return fmaf(b.hi, x, b.lo != 0.0f ? fmaf(b.lo, x, add) : add);
}

// One element of AdamW in fp32; A holds lr, eps and the bias corrections.
template <typename A>
__device__ __forceinline__ void adamw_one(float& p, float g, float& m, float& v, const A& a, const AdamBetas& b,
                                          float wd) {
  m = decayed(b.b1, m, b.b1.rest * g);
  v = decayed(b.b2, v, b.b2.rest * g * g);
  const float mh = m / a.bc1;
  const float vh = v / a.bc2;
  p = p - a.lr * (mh / (sqrtf(vh) + a.eps) + wd * p);
}

// min(1, max_norm / (norm + 1e-6)); a NaN norm gives NaN, an infinite one 0.
__device__ __forceinline__ float clip_coef(const ClipArg& c) {
  if (!c.norm) return 1.0f;
  const float x = c.max_norm / (*c.norm + 1e-6f);
  return x >= 1.0f ? 1.0f : x;
}

}  // namespace muon
