// phs_decay.cuh -- the decay of recurrent states, shared by linear attention
// and the selective scan.
#pragma once

#include "phs_common.cuh"

namespace phs {

// A state's decay over some tokens whose log decays add up to x, as one factor.
// Small ones (-1/2 < x <= 0) as exp(x) - 1, of negative sign, and the state as s +
// factor s: the rounding of exp(x) itself, off by up to 2^-25, would come back in
// every step and grow with the memory of the head (a rate of 2e-4 holds 5,000
// tokens: 1.5e-4 of the state).  Strong ones as exp(x): there the rounding of
// exp(x) - 1, off by up to 2^-25 too, would be more than what is left (10 % of it
// at x = -15).
__device__ __forceinline__ float decay_factor(float x) {
  return x > -0.5f && x <= 0.f ? copysignf(expm1f(x), -1.f) : expf(x);
}
__device__ __forceinline__ bool is_small_decay(float factor) { return signbit(factor); }
__device__ __forceinline__ float decayed(float s, float factor) {
  return fmaf(s, factor, is_small_decay(factor) ? s : 0.f);
}

}  // namespace phs
