// phs_prompt.cuh -- device primitives of the chunked prompt kernels (linear
// attention, the selective scan): waits of limited length shared by a CTA's
// roles, register splits, values as sums of bf16 terms.
#pragma once

#include "phs_pairs.cuh"
#include "phs_tc.cuh"

namespace phs {

// Bounded wait that also gives up when another role has.  (The loop is kept
// small, since the roles' code competes for the instruction caches.)
__device__ __forceinline__ bool lin_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity))
    if (*abort || global_timer_ns() - t0 > kWaitLimitNs) return false;
  return true;
}

// The same by a whole warp, one answer for all its lanes.
__device__ __forceinline__ bool lin_wait_warp(uint32_t bar, uint32_t parity, volatile int* abort) {
  return __all_sync(0xffffffffu, lin_wait(bar, parity, abort));
}

template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// (by fma with bf16 factors, here and below: shifts and masks would run on the
// units that the conversions keep busy)
__device__ __forceinline__ uint64_t f2_bf16(uint32_t w) {
  float lo, hi;
  asm("{\n\t.reg .b16 l, h, m;\n\t"
      "mov.b16 m, 0x3F80;\n\t"  // 1
      "mov.b32 {l, h}, %2;\n\t"
      "fma.rn.f32.bf16 %0, l, m, %3;\n\t"
      "fma.rn.f32.bf16 %1, h, m, %3;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(w), "f"(0.f));
  return f2(lo, hi);
}
// bf16 pair of two values, and with take_term the values keep what it leaves
__device__ __forceinline__ uint32_t pack_term(uint64_t x) {
  const float2 v = f2_get(x);
  return pack_bf16(v.x, v.y);
}
__device__ __forceinline__ uint32_t take_term(uint64_t& x) {
  const float2 v = f2_get(x);
  const uint32_t w = pack_bf16(v.x, v.y);
  float lo, hi;
  asm("{\n\t.reg .b16 l, h, m;\n\t"
      "mov.b16 m, 0xBF80;\n\t"  // -1
      "mov.b32 {l, h}, %2;\n\t"
      "fma.rn.f32.bf16 %0, l, m, %3;\n\t"
      "fma.rn.f32.bf16 %1, h, m, %4;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(w), "f"(v.x), "f"(v.y));
  x = f2(lo, hi);
  return w;
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t x, uint32_t y, uint32_t z,
                                       uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z),
               "r"(w)
               : "memory");
}

// Tensor-memory store in the layout that ldmatrix.trans delivers: 16 lanes,
// 4 N columns; thread 4 r + c holds column 4 i + c of lanes r (word 2 i) and
// r + 8 (word 2 i + 1).  Here N = 2.
__device__ __forceinline__ void tmem_st_16x128(uint32_t taddr, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(x), "r"(y), "r"(src)
      : "memory");
}

}  // namespace phs
