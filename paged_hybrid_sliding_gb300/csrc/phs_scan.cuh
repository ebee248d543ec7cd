// phs_scan.cuh -- what the selective scan's kernels for tokens and for prompts
// share: a request's state and tokens, a token's step.
#pragma once

#include "phs_common.cuh"
#include "phs_decay.cuh"
#include "phs_layers.h"

namespace phs {

// The state of request b, or -1 where it has none: a negative id (an
// inactive request), one outside the pool, or one that an earlier request
// has.  All threads of the CTA call it.
__device__ __forceinline__ int64_t scan_state(const ScanArgs& a, int b) {
  if (!a.state_ids) return b;  // the launcher checked that B <= num_states
  const int id = a.state_ids[b];
  int again = 0;
  for (int j = threadIdx.x; j < b; j += blockDim.x) again |= a.state_ids[j] == id;
  again = __syncthreads_or(again);
  if (id < 0) return -1;
  if (id >= a.num_states || again) {
    if (threadIdx.x == 0) set_status(a.status, again ? PHS_EINVAL : PHS_ERANGE);
    return -1;
  }
  return id;
}

// The step of token t for head h.  (exp(20) + 1 rounds to exp(20) and a little:
// above it softplus is its argument to fp32.)
__device__ __forceinline__ float scan_step(const ScanArgs& a, int64_t t, int h) {
  const int64_t at = t * a.dt_stride + h;
  float x = a.dt_f32 ? reinterpret_cast<const float*>(a.dt)[at]
                     : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(a.dt)[at]);
  if (a.dt_bias) x += a.dt_bias[h];
  return x > 20.f ? x : log1pf(expf(x));
}

// The token range of request b; false where it is bad: outside the tokens,
// longer than stated, or beginning before the end of an earlier one (two
// requests must not write one row).  All threads of the CTA call it.
__device__ __forceinline__ bool scan_tokens(const ScanArgs& a, int b, int& t0, int& t1) {
  t0 = a.cu_seqlens[b];
  t1 = a.cu_seqlens[b + 1];
  int bad = t0 < 0 || t1 < t0 || t1 > a.total_tokens || t1 - t0 > a.max_seq;
  for (int j = threadIdx.x; j < b; j += blockDim.x) bad |= a.cu_seqlens[j] > t0;
  bad = __syncthreads_or(bad);
  if (bad && threadIdx.x == 0) set_status(a.status, PHS_ERANGE);
  return !bad;
}

}  // namespace phs
