// phs_quant.cuh -- from bf16 values to the stored bytes of 8-bit codes, shared
// by the block quantiser and the quantising cache writes.
#pragma once

#include "phs_pairs.cuh"

namespace phs {

// Magic-number rounding: for |y| < 2^22, fl(y + 1.5 * 2^23) rounds y to the
// nearest integer (ties to even, the default rounding) and keeps it in the
// low mantissa bits.  With 128 added to the constant (128 is even, so the
// ties still go to even) the low byte of the sum's bits is the stored byte
// x + 128.
constexpr float kRoundMagicOffset = 12582912.0f + 128.0f;

// The three-input maximum and minimum.
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float fmin3(float a, float b, float c) {
  float r;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Stored bytes of 8 values (bf16 pairs v[0..3]) at scale s, rs2 the pair of
// fl(1 / s) (0 where s is 0), always_divide where that overflows:
// code = rint(x / s) with x / s the IEEE quotient.  y = x * fl(1/s) is
// within |x/s| * (2^-23 + 2^-48) + ulp/2 <= 1.9e-5 of that quotient (|x/s|
// <= 127.5), so rint(y) equals rint(x / s) unless y lies within 1.9e-5 of
// a half-integer: a group of 8 codes holding such an element takes the
// IEEE division for all 8 (rare).  A scale so small that 1/s overflows
// (subnormal groups) always divides.  |rint(x / s)| <= 127 by
// construction, so no clamp is needed.  s == 0 gives rs == 0 and every
// code 0.  The rounding steps run on packed pairs (two elements per
// instruction, each rounded as the scalar operation would be).
__device__ __forceinline__ uint2 quant_codes8(const uint32_t* v, float s, uint64_t rs2,
                                              bool always_divide) {
  const uint64_t magic2 = f2(kRoundMagicOffset, kRoundMagicOffset);
  uint32_t t[8];  // fl(rint(code) + 1.5 * 2^23): the code in the low byte
  float dmax = 0.f, dmin = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    // bf16 pair -> fp32 pair: the bf16 bits are the high half of the fp32
    const uint64_t f = f2(__uint_as_float(v[k] << 16), __uint_as_float(v[k] & 0xFFFF0000u));
    const uint64_t y = f2_mul(f, rs2);
    const uint64_t tt = f2_add(y, magic2);
    const uint64_t d = f2_sub(y, f2_sub(tt, magic2));  // y - rint(y), in [-1/2, 1/2]
    const float2 dd = f2_get(d), tf = f2_get(tt);
    dmax = fmax3(dmax, dd.x, dd.y);
    dmin = fmin3(dmin, dd.x, dd.y);
    t[2 * k] = __float_as_uint(tf.x);
    t[2 * k + 1] = __float_as_uint(tf.y);
  }
  if (always_divide || dmax > 0.4999f || dmin < -0.4999f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float xv = __uint_as_float(e & 1 ? v[e >> 1] & 0xFFFF0000u : v[e >> 1] << 16);
      t[e] = __float_as_uint(__fadd_rn(rintf(__fdiv_rn(xv, s)), kRoundMagicOffset));
    }
  }
  uint32_t w[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t lo = __byte_perm(t[4 * k], t[4 * k + 1], 0x0040);
    const uint32_t hi = __byte_perm(t[4 * k + 2], t[4 * k + 3], 0x0040);
    w[k] = __byte_perm(lo, hi, 0x5410);
  }
  return make_uint2(w[0], w[1]);
}

}  // namespace phs
