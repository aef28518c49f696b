// Device arithmetic shared by the elementwise kernels: the AdamW update of one element and the
// clip coefficient.
#pragma once

#include <hip/hip_runtime.h>

#include "list_types.h"

namespace muon {

// One element of AdamW in fp32; A holds lr, beta1, beta2, eps and the bias corrections.
template <typename A>
__device__ __forceinline__ void adamw_one(float& p, float g, float& m, float& v, const A& a, float wd) {
  m = fmaf(a.beta1, m, (1.0f - a.beta1) * g);
  v = fmaf(a.beta2, v, (1.0f - a.beta2) * g * g);
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
