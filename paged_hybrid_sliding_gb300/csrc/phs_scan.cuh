// phs_scan.cuh -- what the selective scan's kernels for tokens and for prompts
// share: a token's step.
#pragma once

#include "phs_common.cuh"
#include "phs_decay.cuh"
#include "phs_layers.h"
#include "phs_request.cuh"

namespace phs {

// The step of token t for head h.  (exp(20) + 1 rounds to exp(20) and a little:
// above it softplus is its argument to fp32.)
__device__ __forceinline__ float scan_step(const ScanArgs& a, int64_t t, int h) {
  const int64_t at = t * a.dt_stride + h;
  float x = a.dt_f32 ? reinterpret_cast<const float*>(a.dt)[at]
                     : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(a.dt)[at]);
  if (a.dt_bias) x += a.dt_bias[h];
  return x > 20.f ? x : log1pf(expf(x));
}

}  // namespace phs
