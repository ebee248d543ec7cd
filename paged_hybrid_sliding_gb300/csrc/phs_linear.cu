// phs_linear.cu -- linear attention with a decay for each head, over a pool
// of per-request states.
//
//   S_t = exp(g_h) S_{t-1} + k_t v_t^T        (D x D, fp32, one per KV head)
//   o_t = scale q_t^T S_t                     (every query head of the group)
// with g_h <= 0 the head's log decay.
#include "phs_common.cuh"
#include "phs_decay.cuh"
#include "phs_merge.cuh"
#include "phs_ops.h"
#include "phs_prompt.cuh"
#include "phs_request.cuh"

namespace phs {

// One CTA per (request, KV head).  A row of the state (one k index) is D/4
// threads of one float4 each, read, updated and written back in registers; the
// outputs' sums over rows meet in shared memory once.  The step reads and
// writes each state once and computes 2 to 3 operations a byte, so it is bound
// by memory, and small CTAs with many loads in flight carry it: 256 requests of
// 32 heads of 128 (1.07 GB) take 170.1 us, 6.4 TB/s, against 159.4 for those
// bytes at the rate of a plain copy; 2 requests 3.3 us, a launch.
template <int D, int GM>
__global__ void __launch_bounds__(256) phs_linear_decode_kernel(const LinearArgs a) {
  constexpr int TR = D / 4, RT = 256 / TR;  // threads of a row, rows at once
  __shared__ float sq[GM][D], sk[D];
  __shared__ float4 so[RT][TR];
  const int b = blockIdx.x, h = blockIdx.y;
  const int r0 = threadIdx.x / TR, c = threadIdx.x % TR;
  const int64_t id = request_state(a, b);
  const size_t qrow = (static_cast<size_t>(b) * a.Hq + static_cast<size_t>(h) * a.G) * D;
  if (id < 0) {
    for (int e = threadIdx.x; e < a.G * D; e += 256) store_out(a.out, qrow + e, 0.f, a.out_f32);
    return;
  }
  const size_t krow = (static_cast<size_t>(b) * a.Hkv + h) * D;
  for (int e = threadIdx.x; e < a.G * D; e += 256)
    sq[e / D][e % D] = __bfloat162float(a.q[qrow + e]) * a.scale;
  for (int e = threadIdx.x; e < D; e += 256) sk[e] = __bfloat162float(a.k[krow + e]);
  float4 v;
  v.x = __bfloat162float(a.v[krow + 4 * c]);
  v.y = __bfloat162float(a.v[krow + 4 * c + 1]);
  v.z = __bfloat162float(a.v[krow + 4 * c + 2]);
  v.w = __bfloat162float(a.v[krow + 4 * c + 3]);
  const float decay = decay_factor(a.log_decay[h]);
  float4* S = reinterpret_cast<float4*>(a.state + (id * a.Hkv + h) * D * D);
  __syncthreads();
  float4 o[GM];
#pragma unroll
  for (int g = 0; g < GM; ++g) o[g] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int r = r0; r < D; r += RT) {
    float4 s = S[r * TR + c];
    s.x = fmaf(sk[r], v.x, decayed(s.x, decay));
    s.y = fmaf(sk[r], v.y, decayed(s.y, decay));
    s.z = fmaf(sk[r], v.z, decayed(s.z, decay));
    s.w = fmaf(sk[r], v.w, decayed(s.w, decay));
    S[r * TR + c] = s;
#pragma unroll
    for (int g = 0; g < GM; ++g) {
      const float q = g < a.G ? sq[g][r] : 0.f;
      o[g].x = fmaf(q, s.x, o[g].x);
      o[g].y = fmaf(q, s.y, o[g].y);
      o[g].z = fmaf(q, s.z, o[g].z);
      o[g].w = fmaf(q, s.w, o[g].w);
    }
  }
#pragma unroll
  for (int g = 0; g < GM; ++g) {
    if (g >= a.G) break;
    __syncthreads();
    so[r0][c] = o[g];
    __syncthreads();
    if (threadIdx.x < D) {
      float x = 0.f;
      for (int r = 0; r < RT; ++r) x += reinterpret_cast<const float*>(so[r])[threadIdx.x];
      store_out(a.out, qrow + g * D + threadIdx.x, x, a.out_f32);
    }
  }
}

template <int D>
static int launch_linear_decode_t(const LinearArgs& a, cudaStream_t stream) {
  const dim3 grid(a.B, a.Hkv);
  if (a.G == 1)
    phs_linear_decode_kernel<D, 1><<<grid, 256, 0, stream>>>(a);
  else if (a.G <= 4)
    phs_linear_decode_kernel<D, 4><<<grid, 256, 0, stream>>>(a);
  else
    phs_linear_decode_kernel<D, 16><<<grid, 256, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? PHS_OK : PHS_ECUDA;
}

int launch_linear_decode(int D, const LinearArgs& a, cudaStream_t stream) {
  return D == 128 ? launch_linear_decode_t<128>(a, stream) : launch_linear_decode_t<64>(a, stream);
}

// ------------------------------------------------------------- prompts --
// Prompts go in chunks of C = 128 tokens.  With S the state before a chunk,
// rows i, j of the chunk, v rows of it real and pw[n] = exp(g n):
//   O = diag(scale pw[i + 1]) Q S + (scale pw[i - j] Q K^T, j <= i) V
//   S <- pw[v] S + sum_j pw[v - 1 - j] k_j v_j^T
// Four matrix products a chunk (and query head), on the tensor cores:
//   QK = Q K^T     128 x 128 x D   A = Q, B = K                (shared memory)
//   QS = Q S       128 x D x D     A = Q, B = S                (shared memory)
//   PV = P V       128 x D x 128   A = P in tensor memory, B = V
//   KV = K'^T V    D x D x 128     A = K'^T in tensor memory, B = V
// The tokens' decay makes P and K' values of 24 bits, and the state is an
// fp32 one.  They enter as sums of bf16 terms: P and S as two (16 bits of
// each value; one term would put its 2^-9 beside the output's own rounding),
// K' as three (24 bits: the state is kept in fp32 and must stay one), and V
// and Q are exact.  KV is accumulated chunk by chunk from zero and added to
// the state in fp32 registers: the tensor cores' own sums drop the bits
// below the running sum's last one, which over a long memory would pull the
// state down.
//
// One CTA per (segment, KV head, request) walks its chunks in order:
//   warps 0-7   rows of the chunk, two threads a row: scores -> P, the
//               inter-chunk part scaled, the output rows
//   warps 8-15  rows of the state, two threads a row, in registers: state ->
//               two terms in shared memory, K tile -> K'^T terms (by warps 0-7
//               where only sums are formed, which have no rows)
//   warp 16     issues KV
//   warp 17     TMA loads: a ring of K and V tiles, two Q tiles
//   warp 18     TMA stores of the output tiles, in Q's place
//   warp 19     issues QK, QS and PV
// KV is issued before PV: its sum's way into the state then runs beside PV.
// Two warps on each scheduler run each role's code, and its loops are kept
// small: with one warp and everything unrolled, fetching instructions was
// the largest stall (3.1 of 10.7 warp-cycles an instruction).
//
// What bounds it: a chunk at D = 128 takes 3.5 us (6,600 cycles) of a CTA, in
// which it has the tensor cores busy for 55 %, its schedulers issue in 56 %, and
// it moves 128 KB, 2.9 us at an SM's share of HBM.  What is left is the chain
// from one chunk's state to the next one's (terms to shared memory, K' and KV,
// its sum back) and, beside it, scores, P, PV and the rows.  One prompt of
// 32,751 tokens and 32 heads of 128: 315 us (a quarter for the sums of segments)
// against 158 for its bytes; of 32,768 tokens and heads of 64, 211 against 79.  Steps that did not help: six warpgroups instead of five (300
// against 265 us for the rows), other forms of the waits, one arrival for a
// warp instead of its threads' (331 against 321), P's loads a step ahead, terms
// cut off instead of rounded (391 against 348) or rounded by two fma (339
// against 337), K' formed before the wait for its buffer (345 against 337), PV
// not held behind KV (326 against 321), fewer parts of K' for a last chunk (325
// against 310).  Single bf16 terms of P or S would help, and are too coarse.
//
// Where there are fewer (request, KV head) pairs than SMs, prompts are cut
// into segments: a first launch sums up their own states (K and V alone; a
// segment in `nsub` parts, as this launch has fewer CTAs), a small one joins
// these sums into the states that the segments start from, and the last one
// forms the rows.  Where SMs are left, a group's query heads go to several
// CTAs (`ngrp`), each of which forms the states for itself.  As the pool's
// state is overwritten by one of these CTAs, they all start from a copy.
constexpr int kLinC = kLinearChunk;
constexpr int kLinThreads = 640;
// registers a thread: 96 at launch, five warpgroups; 2 x 88 + 2 x 120 + 64 = 5 x 96
constexpr int kLinRegsRows = 88, kLinRegsState = 120, kLinRegsIssue = 64;
// Tensor-memory columns: a chunk's sum U, scores (and P), output, and a ring
// of parts of K'^T: beside the rows at D = 128 parts of 16 tokens, 5 of a
// chunk's 8; else two of 64.  Forming the next parts runs beside the product
// with the last.  (8 prompts of 4,096 tokens, 32 heads of 128: 250 us, against
// 262 with two parts of 32 tokens.  One of 32,768 and heads of 64: 207 us with
// parts of 64, 236 of 32, 261 of 16.)  Where there are no rows U has two
// buffers, and a chunk's KV does not wait for the last one's sum to be taken
// up.
template <int D, bool STATES>
struct LinTmem {
  static constexpr uint32_t kU = 0;
  static constexpr int kUBufs = STATES ? 2 : 1;
  static constexpr uint32_t kOut = D == 64 ? 64 : 256;
  static constexpr uint32_t kSc = 128;
  static constexpr uint32_t kKp = STATES || D == 64 ? 256 : 384;
  static constexpr int kSteps = STATES || D == 64 ? 4 : 1;  // of 16 tokens
  static constexpr uint32_t kPart = 24 * kSteps;  // a step: 3 terms of 8 columns
  static constexpr int kRing = (512 - kKp) / kPart;
  static_assert(kUBufs * D <= kKp, "tensor memory");
};

template <int D, bool STATES>
struct LinLayout {
  static constexpr int kTile = kLinC * D * 2;  // [D / 64 halves][128 rows][128 bytes]
  static constexpr int kHalf = kLinC * 128;
  static constexpr int kSlots = STATES || D == 64 ? 6 : 3;  // K(0) V(0) K(1) V(1) ... in turn
  static constexpr int kKV = 0;
  static constexpr int kQ = kKV + kSlots * kTile;
  // two tiles in turn, each for a pair's Q and then for its output: the next Q
  // is loaded a pair ahead
  static constexpr int kS = kQ + 2 * kTile;    // 2 terms [D / 64][D rows][128 bytes]
  static constexpr int kSTerm = D * D * 2;
  static constexpr int kBar = STATES ? kQ : kS + 2 * kSTerm;
  static constexpr int kBars = 2 * kSlots + 2 * LinTmem<D, STATES>::kRing + 19;
  static constexpr int kMisc = kBar + kBars * 8;  // tensor-memory base, abort flag
  static constexpr int kAlloc = kMisc + 16 + 1024;
  static constexpr int kTables = (3 * kLinC + 4 + 32 + 2) * 4;  // static: back, ps and its pad, factors
  static_assert(kAlloc + kTables <= 227 * 1024, "shared memory of the prompt kernel");
};

// The request that comes `at`-th when the longest come first.  Where there are
// more CTAs than SMs, the last ones to start then end soon: 48.5 us against 61
// for 16 prompts of 1 to 517 tokens, 32 heads on 8.  All threads of the CTA
// call it.
__device__ __forceinline__ int request_by_length(const LinearArgs& a, int at) {
  __shared__ int found;
  static_assert(kLinearSort <= kLinThreads, "a thread for each request");
  const int j = threadIdx.x;
  if (j < a.B) {
    const int64_t len = int64_t{a.cu_seqlens[j + 1]} - a.cu_seqlens[j];
    int before = 0;
    int64_t from = a.cu_seqlens[0];
    for (int i = 0; i < a.B; ++i) {
      const int64_t to = a.cu_seqlens[i + 1];
      before += to - from > len || (to - from == len && i < j);
      from = to;
    }
    if (before == at) found = j;
  }
  __syncthreads();
  return found;
}

// STATES: the first launch (sums of each segment but the last, no outputs)
template <int D, bool STATES>
__global__ void __launch_bounds__(kLinThreads, 1)
    phs_linear_prompt_kernel(const __grid_constant__ CUtensorMap tq,
                             const __grid_constant__ CUtensorMap tk,
                             const __grid_constant__ CUtensorMap tv,
                             const __grid_constant__ CUtensorMap to,
                             const __grid_constant__ LinearArgs a) {
  using L = LinLayout<D, STATES>;
  using T = LinTmem<D, STATES>;
  constexpr uint32_t kTmU = T::kU, kTmSc = T::kSc, kTmOut = T::kOut, kTmKp = T::kKp;
  constexpr int kTermWarps = 2;  // that form K' of 32 columns of K
  constexpr int kTermThreads = 128 * kTermWarps;
  constexpr int kBefore = D == 64 ? 1 : 0;  // parts of a warp before the state, see below
  extern __shared__ uint8_t smem_raw[];
  // back[x]: the decay of token x of a whole chunk up to its last one, exp(g
  // (127 - x)), then zeros for tokens behind the last; ps[n] = scale exp(g n),
  // read from n = -31 on (unused there)
  __shared__ float back[2 * kLinC], ps_pad[32 + kLinC + 4];
  __shared__ float factors[2];  // decay factors of a whole chunk and of the last one
  const float* ps = ps_pad + 32;
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // (known to be uniform)
  // part: the segment's first one, with STATES the one to sum up
  int b = blockIdx.x, h = blockIdx.y, part = blockIdx.z, grp = 0;
  if (!STATES) {
    const int of_b = a.Hkv * a.nseg * a.ngrp, i = blockIdx.x % of_b;
    b = blockIdx.x / of_b;
    h = i % a.Hkv;
    part = i / a.Hkv / a.ngrp * a.nsub;
    grp = i / a.Hkv % a.ngrp;
    if (a.longest_first) b = request_by_length(a, b);
  }
  const int G = a.G / a.ngrp;
  const int head0 = h * a.G + grp * G;  // first of this CTA's query heads

  if (STATES) pdl_launch_dependents();  // the join waits for this grid's end

  // ---- this CTA's chunks
  const int64_t id = request_state(a, b);
  int t0, t1;
  if (!request_tokens(a, b, t0, t1)) {
    pdl_wait_prior_grid();
    return;
  }
  const int all = (t1 - t0 + kLinC - 1) / kLinC, parts = a.nseg * a.nsub;
  const int next = part + (STATES ? 1 : a.nsub);
  const bool last = next == parts;
  const int c0 = part_chunk(a, all, part), c1 = part_chunk(a, all, next);
  if (c0 == c1 && !last) {
    pdl_wait_prior_grid();
    return;
  }
  t1 = min(t1, t0 + c1 * kLinC);
  t0 += c0 * kLinC;
  if (id < 0) {  // no state: zero rows
    if (!STATES)
      for (int64_t e = tid; e < static_cast<int64_t>(t1 - t0) * G * D; e += kLinThreads) {
        const int64_t t = t0 + e / (G * D);
        reinterpret_cast<__nv_bfloat16*>(a.out)[(t * a.Hq + head0) * D + e % (G * D)] =
            __float2bfloat16_rn(0.f);
      }
    pdl_wait_prior_grid();
    return;
  }
  const int nch = (t1 - t0 + kLinC - 1) / kLinC;
  const float g0 = a.log_decay[h], g = g0 < -1e4f ? -1e4f : g0;  // exp(g n) is 0 there anyway

  // barriers: tile loaded / used, Q, scores, the inter-chunk part, P and that
  // part ready, output complete / read, K' terms written / used, state (the
  // last chunk's sum is read, the state's terms written, V's rows behind the
  // last token zero), chunk sum complete, output tile written / stored, all
  // of a chunk's KV issued, its last PV issued
  auto bar = [sb](int i) { return sb + L::kBar + 8 * i; };
  constexpr int kB = 2 * L::kSlots;
  const uint32_t kv_full = bar(0), kv_empty = bar(L::kSlots), q_full = bar(kB),
                 y_full = bar(kB + 2), y_free = bar(kB + 4), s_ready = bar(kB + 6),
                 u_done = bar(kB + 8), drain = bar(kB + 10), sc_full = bar(kB + 12),
                 qs_done = bar(kB + 13), pv_ready = bar(kB + 14), o_done = bar(kB + 15),
                 o_free = bar(kB + 16), kv_all = bar(kB + 17), pv_issued = bar(kB + 18),
                 kp_full = bar(kB + 19), kp_empty = bar(kB + 19 + T::kRing);
  static_assert(kB + 19 + 2 * T::kRing == L::kBars, "barriers (the first six: pairs)");
  volatile int* abort = reinterpret_cast<volatile int*>(smem + L::kMisc + 4);
  if (warp == 16) {
    tmem_alloc(sb + L::kMisc, 512);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < L::kSlots; ++i) {
      mbar_init(kv_full + 8 * i, 1);
      // the threads that form K' and, of a V tile, the products KV and PV; of a
      // K tile, QK and one of those threads again
      mbar_init(kv_empty + 8 * i, kTermThreads + (STATES ? 1 : 2));
    }
    for (int i = 0; i < T::kRing; ++i) {
      mbar_init(kp_full + 8 * i, 128);
      mbar_init(kp_empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + 8 * i, 1);
      mbar_init(y_full + 8 * i, 256);
      mbar_init(y_free + 8 * i, 1);
    }
    mbar_init(sc_full, 1);
    mbar_init(qs_done, 1);
    mbar_init(pv_ready, 256);
    mbar_init(o_done, 1);
    mbar_init(o_free, 256);
    for (int i = 0; i < T::kUBufs; ++i) {
      mbar_init(s_ready + 8 * i, 256);
      mbar_init(u_done + 8 * i, STATES ? 1 : 2);  // KV, and QS done with the state's terms
    }
    mbar_init(kv_all, 1);
    mbar_init(pv_issued, 1);
    mbar_init(drain, 1);
    mbar_init(drain + 8, 1);
    *abort = 0;
    fence_mbar_init();
  }
  for (int n = tid; n <= kLinC; n += kLinThreads) {
    const float p = expf(g * n);
    if (n < kLinC) {
      back[kLinC - 1 - n] = p;
      back[kLinC + n] = 0.f;
    }
    ps_pad[32 + n] = p * a.scale;
    if (n < 32) ps_pad[n] = 0.f;
  }
  // (by threads that have no part in the tables)
  if (tid == 160) factors[0] = decay_factor(g * kLinC);
  if (tid == 192) factors[1] = decay_factor(g * (t1 - t0 - (nch - 1) * kLinC));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem =
      __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(smem + L::kMisc), 0);
  const uint32_t my_lanes = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);

  // parts of a chunk whose places in the ring are free when the state is there
  constexpr int kKnownFree = !STATES && kBefore == 0 ? T::kRing : 0;

  // ---- K'^T of 32 columns of K, as three terms: ldmatrix.trans gives thread
  // 4 x + y tokens 2 y, 2 y + 1 (of 8) of column x of each of 4 groups of 8
  // columns.  The kTermWarps warps of these columns, of which this is number
  // `which`, take parts in turn.  `between(n)` is called before the first of
  // them, at D = 64 after it (the state is what the others wait for: 327 us for
  // 32,751 tokens of 32 heads, 348 after the first; but 230 and 211 at 64).
  auto form_terms = [&](int which, auto&& between) {
    const int qt = warp & 3, kx = lane >> 3;  // matrix kx: columns 32 qt + 8 kx ..
    const bool mine = 32 * qt < D;            // D = 64: the upper half has no columns
    const uint32_t kcol = (qt >> 1) * L::kHalf + (lane & 7) * 128 +
                          ((((4 * (qt & 1) + kx) ^ lane) & 7) << 4);
    if (!mine && which == 0) {  // rows 64..127 of K'^T are zero
      uint32_t z[16];
#pragma unroll
      for (int c = 0; c < 16; ++c) z[c] = 0u;
      static_assert(D == 128 || T::kRing * T::kPart % 16 == 0, "in stores of 16 columns");
      for (uint32_t c = 0; c < T::kRing * T::kPart; c += 16) tmem_st16(my_lanes + kTmKp + c, z);
      tmem_st_wait();
    }
    bool ok = true;
    int place = which, turn = 0;  // in the ring, of this warp's next part
    for (int n = 0; ok && n < nch; ++n) {
      const int v = min(kLinC, t1 - t0 - n * kLinC);
      const int ki = 2 * n, vi = 2 * n + 1;  // tiles of the ring
      const uint32_t kt = sb + L::kKV + (ki % L::kSlots) * L::kTile;
      const float* decay = back + kLinC - v + 2 * (lane & 3);  // of this thread's two tokens
      ok = lin_wait_warp(kv_full + 8 * (ki % L::kSlots), (ki / L::kSlots) & 1, abort);
      if (!ok) break;
      if (v < kLinC) {
        // rows behind the last token: no 0 * NaN.  K: what this warp reads
        // itself, its own parts' rows, since nothing orders it with the others
        // here (QK may read either; those scores are masked); V: all.
        ok = lin_wait_warp(kv_full + 8 * (vi % L::kSlots), (vi / L::kSlots) & 1, abort);
        if (!ok) break;
        const uint32_t vt = sb + L::kKV + (vi % L::kSlots) * L::kTile;
        for (int t = v + (lane >> 2); mine && t < kLinC; t += 8)
          if (t / (16 * T::kSteps) % kTermWarps == which)
            sts128(kt + (qt >> 1) * L::kHalf + t * 128 +
                       ((((4 * (qt & 1) + (lane & 3)) ^ t) & 7) << 4),
                   0, 0, 0, 0);
        for (int u = 128 * which + 32 * qt + lane; u < D / 64 * (kLinC - v) * 8;
             u += kTermThreads) {
          const int hf = u / ((kLinC - v) * 8), x = u % ((kLinC - v) * 8);
          sts128(vt + hf * L::kHalf + v * 128 + x * 16, 0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
      constexpr int kParts = kLinC / 16 / T::kSteps;
#pragma unroll 1
      for (int p = which; ok && p < kParts + kTermWarps; p += kTermWarps) {
        if (p / kTermWarps == kBefore) ok = between(n);
        if (!ok || p >= kParts) break;
        // (a wait costs 100 cycles even where it has nothing to wait for: what
        // the last chunk had in the ring is known to be read once its sum is there)
        if (turn > 0 && p >= kKnownFree)
          ok = lin_wait_warp(kp_empty + 8 * place, (turn - 1) & 1, abort);
        if (!ok) break;
        tc_fence_after();
        if (mine) {
#pragma unroll
          for (int st = 0; st < T::kSteps; ++st) {
            const int t = 16 * (T::kSteps * p + st);  // first token
            uint32_t w[3][2][4];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              uint32_t k[4];
              ldsm_x4_t(kt + kcol + (t + 8 * q) * 128, k[0], k[1], k[2], k[3]);
              const uint64_t f = f2(decay[t + 8 * q], decay[t + 8 * q + 1]);
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                uint64_t y = f2_mul(f2_bf16(k[x]), f);
                w[2][x >> 1][2 * q + (x & 1)] = take_term(y);
                w[1][x >> 1][2 * q + (x & 1)] = take_term(y);
                w[0][x >> 1][2 * q + (x & 1)] = pack_term(y);
              }
            }
#pragma unroll
            for (int i = 0; i < 3; ++i)
#pragma unroll
              for (int x = 0; x < 2; ++x)
                tmem_st_16x128(my_lanes + (static_cast<uint32_t>(16 * x) << 16) + kTmKp +
                                   T::kPart * place + 24 * st + 8 * i,
                               w[i][x]);
          }
          tmem_st_wait();
        }
        tc_fence_before();
        mbar_arrive(kp_full + 8 * place);
        if ((place += kTermWarps) >= T::kRing) {
          place -= T::kRing;
          ++turn;
        }
      }
      // V's place in the ring was an earlier K's: only once V is there do all of
      // that tile's users have let go of it, and an arrival counts for V (a warp
      // that is ahead of the others would else take part in the wrong phase)
      ok = ok && lin_wait_warp(kv_full + 8 * (vi % L::kSlots), (vi / L::kSlots) & 1, abort);
      if (!ok) break;
      mbar_arrive(kv_empty + 8 * (ki % L::kSlots));
      if (which == 0 && qt == 0 && lane == 0) mbar_arrive(kv_empty + 8 * (ki % L::kSlots));
      mbar_arrive(kv_empty + 8 * (vi % L::kSlots));
    }
    return ok;
  };

  // The first tiles are on their way while an earlier launch ends; all else
  // waits for that end here, not in a wait of limited length.
  if (!STATES && warp != 17) pdl_wait_prior_grid();

  // (each warpgroup sets its registers at the head of its own branch, so that
  // the code behind it is compiled for that number)
  if (warp >= 16) {
    regs_dec<kLinRegsIssue>();
    if (warp == 17) {
      // ---------------------------------------------------------------- TMA
      if (lane == 0 && nch > 0) {
        prefetch_tmap(&tk);
        prefetch_tmap(&tv);
        if (!STATES) prefetch_tmap(&tq);
        const uint64_t pol = policy_evict_first();
        auto load = [&](const CUtensorMap* map, uint32_t dst, int head, int t, uint32_t bar) {
          for (int hf = 0; hf < D / 64; ++hf)
            tma_load_2d(dst + hf * (kLinC * 128), map, head * D + 64 * hf, t, bar, pol);
        };
        bool ok = true;
        int nq = 0, tiles = 0;  // Q tiles, K and V tiles issued
        auto load_kv = [&](const CUtensorMap* map, int t) {
          const int slot = tiles % L::kSlots, turn = tiles / L::kSlots;
          if (turn > 0) ok = ok && lin_wait(kv_empty + 8 * slot, (turn - 1) & 1, abort);
          if (!ok) return;
          mbar_arrive_expect_tx(kv_full + 8 * slot, L::kTile);
          load(map, sb + L::kKV + slot * L::kTile, h, t, kv_full + 8 * slot);
          ++tiles;
        };
        auto load_q = [&](int gq, int t) {
          const int at = nq & 1;
          if (nq >= 2) ok = ok && lin_wait(y_free + 8 * at, ((nq >> 1) - 1) & 1, abort);
          if (!ok) return;
          mbar_arrive_expect_tx(q_full + 8 * at, L::kTile);
          load(&tq, sb + L::kQ + at * L::kTile, head0 + gq, t, q_full + 8 * at);
          ++nq;
        };
        for (int n = 0; ok && n < nch; ++n) {
          const int t = t0 + n * kLinC;
          load_kv(&tk, t);
          if (!STATES && ok) load_q(0, t);
          if (ok) load_kv(&tv, t);
          if (!STATES && n == 0) pdl_wait_prior_grid();
          for (int gq = 1; !STATES && ok && gq < G; ++gq) load_q(gq, t);
        }
        if (!ok) {
          set_status(a.status, PHS_ETIMEOUT);
          *abort = 1;
        }
        // copies still in flight land before the CTA ends
        for (int i = max(0, tiles - L::kSlots); i < tiles; ++i)
          (void)mbar_wait(kv_full + 8 * (i % L::kSlots), (i / L::kSlots) & 1);
        for (int i = max(0, nq - 2); i < nq; ++i)
          (void)mbar_wait(q_full + 8 * (i & 1), (i >> 1) & 1);
      }
    } else if (warp == 16 || (!STATES && warp == 19)) {
      // ----------------------------------------------------------- products
      // A whole warp walks the chunks and one elected lane issues: what the
      // instructions take is then known to be the same in every lane, and the
      // compiler keeps it in uniform registers (issued from a lane of its own,
      // an instruction took 90 cycles and more, whatever its width).
      constexpr uint32_t kIdQK = idesc_bf16_f32(128, kLinC, false, false);
      constexpr uint32_t kIdD = idesc_bf16_f32(128, D, false, true);
      bool ok = true;
      const bool lead = elect_one();
      auto wait = [&](uint32_t bar, int turn) {
        ok = ok && lin_wait_warp(bar, turn & 1, abort);
      };
      // tile i of the ring: its place, once it has been loaded
      auto tile = [&](int i) { return sb + L::kKV + (i % L::kSlots) * L::kTile; };
      auto tile_full = [&](int i) { wait(kv_full + 8 * (i % L::kSlots), i / L::kSlots); };
      auto tile_empty = [&](int i) { return kv_empty + 8 * (i % L::kSlots); };
      if (warp == 16) {  // KV
        int place = 0, turn = 0;  // of the next part of K'
        for (int n = 0; ok && n < nch; ++n) {
          const int ub = n % T::kUBufs;
          tile_full(2 * n + 1);
          if (!STATES)
            wait(s_ready, n);
          else if (n >= 2)  // the sum two chunks ago has been taken up
            wait(s_ready + 8 * ub, n / 2 - 1);
          uint64_t v = sdesc_sw128(tile(2 * n + 1), L::kHalf, 1024);
#pragma unroll 1
          for (int p = 0; p < kLinC / 16; p += T::kSteps, v += T::kSteps * 2048 >> 4) {
            wait(kp_full + 8 * place, turn);
            if (!ok) break;
            tc_fence_after();
            if (lead) {
              const uint32_t kp = tmem + kTmKp + T::kPart * place;
#pragma unroll
              for (int t = 0; t < 3; ++t)
#pragma unroll
                for (int st = 0; st < T::kSteps; ++st)
                  umma_bf16_ts(tmem + kTmU + D * ub, kp + 24 * st + 8 * t, v + (st * 2048 >> 4),
                               kIdD, p > 0 || t > 0 || st > 0);
              umma_commit(kp_empty + 8 * place);
            }
            __syncwarp();
            if (++place == T::kRing) {
              place = 0;
              ++turn;
            }
          }
          // (the other warp has issued the last chunk's PV, so it has waited for
          // that chunk's phase)
          if (!STATES && n >= 1) wait(pv_issued, n - 1);
          if (ok && lead) {
            if (!STATES) mbar_arrive(kv_all);
            umma_commit(u_done + 8 * ub);
            umma_commit(tile_empty(2 * n + 1));
          }
          __syncwarp();
        }
      } else {  // QK, QS, PV
        // (for 32,751 tokens: 323 us at 4, 327 at 2; at D = 64 213 and 207)
        constexpr int kIssue = D == 64 ? 2 : 4;
        // descriptors; a later part of a tile is `bytes >> 4` further on
        const uint64_t dq0 = sdesc_sw128(sb + L::kQ, 16, 1024);
        const uint64_t ds = sdesc_sw128(sb + L::kS, D * 128, 1024);
        int pair = 0;
        for (int n = 0; ok && n < nch; ++n)
          for (int gq = 0; ok && gq < G; ++gq, ++pair) {
            const bool last = gq == G - 1;
            if (gq == 0) tile_full(2 * n);
            wait(q_full + 8 * (pair & 1), pair >> 1);
            const uint64_t dq = dq0 + (pair & 1) * (L::kTile >> 4);
            if (pair >= 1) wait(o_done, pair - 1);  // P of the last pair is read
            if (!ok) break;
            tc_fence_after();
            const uint64_t k = sdesc_sw128(tile(2 * n), 16, 1024);
            if (lead) {
#pragma unroll kIssue
              for (int ks = 0; ks < D / 16; ++ks) {
                const uint32_t at = ((ks >> 2) * L::kHalf + (ks & 3) * 32) >> 4;
                umma_bf16(tmem + kTmSc, dq + at, k + at, kIdQK, ks > 0);
              }
              umma_commit(sc_full);
              if (last) umma_commit(tile_empty(2 * n));
            }
            __syncwarp();
            if (gq == 0) wait(s_ready, n);
            if (pair >= 1) wait(o_free, pair - 1);
            if (!ok) break;
            tc_fence_after();
            if (lead) {
#pragma unroll 1
              for (int t = 0; t < 2; ++t)
#pragma unroll kIssue
                for (int ks = 0; ks < D / 16; ++ks)
                  umma_bf16(tmem + kTmOut, dq + (((ks >> 2) * L::kHalf + (ks & 3) * 32) >> 4),
                            ds + ((t * L::kSTerm + ks * 2048) >> 4), kIdD, t > 0 || ks > 0);
              umma_commit(qs_done);
              if (last) umma_commit(u_done);  // the state's terms have been read
            }
            __syncwarp();
            if (gq == 0) tile_full(2 * n + 1);
            if (last) wait(kv_all, n);
            wait(pv_ready, pair);
            if (!ok) break;
            tc_fence_after();
            const uint64_t v = sdesc_sw128(tile(2 * n + 1), L::kHalf, 1024);
            if (lead) {
#pragma unroll 1
              for (int t = 0; t < 2; ++t)
#pragma unroll kIssue
                for (int ks = 0; ks < kLinC / 16; ++ks)
                  umma_bf16_ts(tmem + kTmOut, tmem + kTmSc + 16 * ks + 8 * t, v + (ks * 2048 >> 4),
                               kIdD, 1u);
              umma_commit(o_done);
              if (last) {
                umma_commit(tile_empty(2 * n + 1));
                mbar_arrive(pv_issued);
              }
            }
            __syncwarp();
          }
      }
      if (!ok && lane == 0) {
        set_status(a.status, PHS_ETIMEOUT);
        *abort = 1;
      }
      // every product of this warp is complete before tensor memory is released
      const uint32_t done = warp == 16 ? drain : drain + 8;
      if (lead) umma_commit(done);
      (void)mbar_wait(done, 0);
      __syncwarp();
    } else if (warp == 18) {
      // --------------------------------------------- whole output tiles out
      if (!STATES && lane == 0) {
        const int whole = (t1 - t0) / kLinC * G;  // (the others' rows are stored by the threads)
        bool ok = true;
        for (int p = 0; ok && p < nch * G; ++p) {
          ok = lin_wait(y_full + 8 * (p & 1), (p >> 1) & 1, abort);
          if (!ok) break;
          if (p < whole) {
            for (int hf = 0; hf < D / 64; ++hf)
              tma_store_2d(&to, sb + L::kQ + (p & 1) * L::kTile + hf * L::kHalf,
                           (head0 + p % G) * D + 64 * hf, t0 + p / G * kLinC);
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
          }
          mbar_arrive(y_free + 8 * (p & 1));
        }
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        if (!ok) {
          set_status(a.status, PHS_ETIMEOUT);
          *abort = 1;
        }
      }
    }
  } else if (!STATES && warp < 8) {
    // ------------------------------------------------- rows of the chunk
    regs_dec<kLinRegsRows>();
    const int qt = warp & 3, half = warp >> 2, i = 32 * qt + lane;  // row
    uint64_t col[8];  // exp(g (15 - e))
#pragma unroll
    for (int e = 0; e < 8; ++e) col[e] = f2(back[112 + 2 * e], back[113 + 2 * e]);
    bool ok = true;
    int pair = 0;
    for (int n = 0; ok && n < nch; ++n)
      for (int gq = 0; ok && gq < G; ++gq, ++pair) {
        ok = lin_wait_warp(sc_full, pair & 1, abort);
        if (!ok) break;
        tc_fence_after();
        // P in place of the scores: 16 columns j of a step of the product
        // become 8 of term 0 and 8 of term 1
#pragma unroll 1
        for (int st = half; st < kLinC / 16; st += 2) {
          uint32_t p[16];
          const int d = i - 16 * st;
          if (st > 2 * qt + 1) {  // behind every row of the warp
#pragma unroll
            for (int e = 0; e < 16; ++e) p[e] = 0u;
          } else {
            uint32_t sc[16];
            tmem_ld16(my_lanes + kTmSc + 16 * st, sc);
            tmem_ld_wait();
            if (st < 2 * qt) {  // before every row: exp(g (d - 15)) exp(g (15 - e))
              const float rf = ps[d - 15];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                uint64_t x = f2_mul(f2_mul(f2(sc[2 * e], sc[2 * e + 1]), f2(rf, rf)), col[e]);
                p[e] = take_term(x);
                p[8 + e] = pack_term(x);
              }
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float y0 = __uint_as_float(sc[2 * e]) * ps[d - 2 * e];
                const float y1 = __uint_as_float(sc[2 * e + 1]) * ps[d - 2 * e - 1];
                uint64_t x = f2(d >= 2 * e ? y0 : 0.f, d >= 2 * e + 1 ? y1 : 0.f);
                p[e] = take_term(x);
                p[8 + e] = pack_term(x);
              }
            }
          }
          tmem_st16(my_lanes + kTmSc + 16 * st, p);
        }
        // the part before the chunk, scaled in place
        ok = lin_wait_warp(qs_done, pair & 1, abort);
        if (!ok) break;
        tc_fence_after();
        const float f = ps[i + 1];
#pragma unroll 1
        for (int c = half * (D / 64); c < (half + 1) * (D / 64); ++c) {
          uint32_t o[32];
          tmem_ld32(my_lanes + kTmOut + 32 * c, o);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 x = f2_get(f2_mul(f2(o[e], o[e + 1]), f2(f, f)));
            o[e] = __float_as_uint(x.x);
            o[e + 1] = __float_as_uint(x.y);
          }
          tmem_st32(my_lanes + kTmOut + 32 * c, o);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(pv_ready);
        // output row: a whole chunk's goes through shared memory and TMA; the
        // rows behind a last token are another request's
        const int t = t0 + n * kLinC + i;
        const bool whole = t0 + (n + 1) * kLinC <= t1;
        ok = lin_wait_warp(o_done, pair & 1, abort);
        if (!ok) break;
        tc_fence_after();
        const uint32_t row = sb + L::kQ + (pair & 1) * L::kTile + i * 128;
        uint4* to_row = reinterpret_cast<uint4*>(
            reinterpret_cast<__nv_bfloat16*>(a.out) +
            (static_cast<size_t>(t) * a.Hq + head0 + gq) * D);
#pragma unroll 1
        for (int c = half * (D / 64); c < (half + 1) * (D / 64); ++c) {
          uint32_t o[32], y[16];
          tmem_ld32(my_lanes + kTmOut + 32 * c, o);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 16; ++e)
            y[e] = pack_bf16(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int u = 4 * c + k;  // 16 bytes of the row
            if (whole)
              sts128(row + (u >> 3) * L::kHalf + (((u ^ i) & 7) << 4), y[4 * k], y[4 * k + 1],
                     y[4 * k + 2], y[4 * k + 3]);
            else if (t < t1)
              to_row[u] = make_uint4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
          }
        }
        tc_fence_before();
        mbar_arrive(o_free);
        if (whole) fence_proxy_async_smem();
        mbar_arrive(y_full + 8 * (pair & 1));
      }
    if (!ok) {
      set_status(a.status, PHS_ETIMEOUT);
      *abort = 1;
    }
  } else if (STATES && warp < 8) {
    regs_dec<kLinRegsRows>();
    if (!form_terms(warp >> 2, [](int) { return true; })) {
      set_status(a.status, PHS_ETIMEOUT);
      *abort = 1;
    }
  } else {
    // ------------------------------------------------- rows of the state
    regs_inc<kLinRegsState>();
    constexpr int N = D / 2;  // columns of a thread
    const int qt = warp & 3, half = (warp >> 2) & 1;
    const int r = 32 * qt + lane;  // row (a k index); D = 64: the upper half has none
    const bool mine = r < D;
    const size_t row = static_cast<size_t>(r) * D + half * N;
    float* pool = a.state + (id * a.Hkv + h) * D * D + row;
    float* ws = a.ws + (static_cast<size_t>(b) * a.Hkv + h) * parts * D * D + row;
    const bool resume = a.resume != nullptr && a.resume[b] != 0;
    uint64_t S[N / 2];  // pairs
#pragma unroll
    for (int c = 0; c < N / 2; ++c) S[c] = 0ull;
    auto store_row = [&](float* to) {
#pragma unroll
      for (int c = 0; c < N; c += 4) {
        const float2 x = f2_get(S[c / 2]), y = f2_get(S[c / 2 + 1]);
        *reinterpret_cast<float4*>(to + c) = make_float4(x.x, x.y, y.x, y.y);
      }
    };
    if (mine && !STATES && (part > 0 || resume)) {
      const float* from = a.nseg > 1 || a.ngrp > 1 ? ws + part * D * D : pool;
#pragma unroll
      for (int c = 0; c < N; c += 4) {
        const float4 x = *reinterpret_cast<const float4*>(from + c);
        S[c / 2] = f2(x.x, x.y);
        S[c / 2 + 1] = f2(x.z, x.w);
      }
    }
    bool ok = true;
    const float chunk_decay = factors[0], last_decay = factors[1];
    // S <- state after chunk n (n >= 0), and where `terms` its two terms to
    // shared memory for the next chunk's QS (the last one has read its own
    // by then: the chunk's sum was issued after it)
    auto next_state = [&](int n, bool terms) {
      const int ub = n >= 0 ? n % T::kUBufs : 0;
      const float d = n == nch - 1 ? last_decay : chunk_decay;
      const uint64_t factor = f2(d, d);
      const float one = is_small_decay(d) ? 1.f : 0.f;
      const uint64_t base = f2(one, one);
      if (n >= 0) {
        ok = ok && lin_wait_warp(u_done + 8 * ub, n / T::kUBufs & 1, abort);
        if (!ok) return;
        tc_fence_after();
      }
      if (mine) {
        const uint32_t my_row = sb + L::kS + r * 128;
#pragma unroll
        for (int c = 0; c < N / 32; ++c) {
          if (n >= 0) {
            uint32_t u[32];
            tmem_ld32(my_lanes + kTmU + D * ub + half * N + 32 * c, u);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e)
              // (the first is a shorter way from the sum to the state, the second
              // fewer instructions: 311 and 317 us for 32,751 tokens of 32 heads of
              // 128, 213 and 210 at 64)
              if constexpr (D == 128)
                S[16 * c + e] = f2_add(f2_fma(S[16 * c + e], factor, f2_mul(S[16 * c + e], base)),
                                       f2(u[2 * e], u[2 * e + 1]));
              else
                S[16 * c + e] = f2_fma(S[16 * c + e], factor,
                                       f2_fma(S[16 * c + e], base, f2(u[2 * e], u[2 * e + 1])));
          }
          if (terms) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t hi[4], lo[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint64_t x = S[16 * c + 4 * k + e];
                hi[e] = take_term(x);
                lo[e] = pack_term(x);
              }
              const int u = half * (N / 8) + 4 * c + k;  // 16 bytes of the row
              const uint32_t at = my_row + (u >> 3) * (D * 128) + (((u ^ r) & 7) << 4);
              sts128(at, hi[0], hi[1], hi[2], hi[3]);
              sts128(at + L::kSTerm, lo[0], lo[1], lo[2], lo[3]);
            }
          }
        }
        if (terms) fence_proxy_async_smem();
      }
      tc_fence_before();
      mbar_arrive(s_ready + 8 * ub);
    };
    if (STATES) {
      for (int n = 0; ok && n < nch; ++n) next_state(n, false);
    } else {
      ok = form_terms(half, [&](int n) {
        next_state(n - 1, true);
        return ok;
      });
      if (nch > 0) next_state(nch - 1, false);
    }
    if (!ok) {
      set_status(a.status, PHS_ETIMEOUT);
      *abort = 1;
    } else if (mine && (STATES || (last && grp == 0))) {
      store_row(STATES ? ws + part * D * D : pool);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 16) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Sums of parts -> the states that segments start from, in the place of their
// first part's: a thread holds 4 elements of a state and walks the parts, 8
// loads at once.  (Joined by each segment for itself instead, a state cost
// it 2.2 us: one prompt of 32,768 tokens, 8 heads on one, 139 us against 76.)
// 8 us for 12 parts of 32 heads.
__global__ void __launch_bounds__(128) phs_linear_join_kernel(const LinearArgs a, int vecs) {
  const int b = blockIdx.x, h = blockIdx.y;
  pdl_launch_dependents();
  const int64_t id = request_state(a, b);
  int t0, t1;
  const bool good = request_tokens(a, b, t0, t1) && id >= 0;
  const int chunks = good ? (t1 - t0 + kLinC - 1) / kLinC : 0, parts = a.nseg * a.nsub;
  const int small = chunks / parts, rest = chunks % parts;  // a part: so many chunks, or one more
  const float g0 = a.log_decay[h], g = g0 < -1e4f ? -1e4f : g0;
  const float decay0 = decay_factor(g * (small * kLinC));
  const float decay1 = decay_factor(g * ((small + 1) * kLinC));
  pdl_wait_prior_grid();
  if (!good) return;
  if (parts == 1) {  // nothing to join: a copy for the groups of heads, 4 loads at once
    if (!a.resume || a.resume[b] == 0) return;
    const float4* from = reinterpret_cast<const float4*>(a.state) + (id * a.Hkv + h) * vecs;
    float4* to = reinterpret_cast<float4*>(a.ws) + (static_cast<size_t>(b) * a.Hkv + h) * vecs;
    const int i0 = blockIdx.z * 512 + threadIdx.x;
    float4 x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = from[i0 + 128 * j];
#pragma unroll
    for (int j = 0; j < 4; ++j) to[i0 + 128 * j] = x[j];
    return;
  }
  const int i = blockIdx.z * 128 + threadIdx.x;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (a.resume && a.resume[b] != 0)
    s = reinterpret_cast<const float4*>(a.state)[(id * a.Hkv + h) * vecs + i];
  float4* at = reinterpret_cast<float4*>(a.ws) +
               (static_cast<size_t>(b) * a.Hkv + h) * parts * vecs + i;
  const int sums = parts - a.nsub;  // the last segment has none
  int frac = 0, sub = 0;            // part_chunk's fraction; number of the part in its segment
  for (int n = 0; n <= sums; n += 8) {
    float4 x[8];
    bool more[8], sum[8];  // of small + 1 chunks; not empty
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      frac += rest;
      more[j] = frac >= parts;
      if (more[j]) frac -= parts;
      sum[j] = n + j < sums && (small > 0 || more[j]);
      if (sum[j]) x[j] = at[static_cast<size_t>(n + j) * vecs];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (n + j <= sums && sub == 0) at[static_cast<size_t>(n + j) * vecs] = s;
      if (++sub == a.nsub) sub = 0;
      if (sum[j]) {
        const float k = more[j] ? decay1 : decay0;
        s = make_float4(decayed(s.x, k) + x[j].x, decayed(s.y, k) + x[j].y,
                        decayed(s.z, k) + x[j].z, decayed(s.w, k) + x[j].w);
      }
    }
  }
}

template <int D>
static int launch_linear_prompt_t(const CUtensorMap& tq, const CUtensorMap& tk,
                                  const CUtensorMap& tv, const CUtensorMap& to,
                                  const LinearArgs& a, cudaStream_t stream) {
  constexpr int kStates = LinLayout<D, true>::kAlloc, kRows = LinLayout<D, false>::kAlloc;
  auto states = phs_linear_prompt_kernel<D, true>;
  auto rows = phs_linear_prompt_kernel<D, false>;
  if (ensure_dynamic_smem(reinterpret_cast<const void*>(rows), kRows) != PHS_OK ||
      ensure_dynamic_smem(reinterpret_cast<const void*>(states), kStates) != PHS_OK)
    return PHS_ECUDA;
  // The launches after the first may start before the one in front of them has
  // ended (they wait for it where they read what it wrote).
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = stream;
  cfg.attrs = &early;
  cudaError_t err = cudaSuccess;
  if (a.nseg > 1) {
    cfg.gridDim = dim3(a.B, a.Hkv, (a.nseg - 1) * a.nsub);
    cfg.blockDim = dim3(kLinThreads);
    cfg.dynamicSmemBytes = kStates;
    err = cudaLaunchKernelEx(&cfg, states, tq, tk, tv, to, a);
    cfg.numAttrs = 1;
  }
  if (err == cudaSuccess && (a.nseg > 1 || (a.ngrp > 1 && a.resume))) {
    cfg.gridDim = dim3(a.B, a.Hkv, D * D / (a.nseg > 1 ? 512 : 2048));  // (1 or 4 vectors a thread)
    cfg.blockDim = dim3(128);
    cfg.dynamicSmemBytes = 0;
    err = cudaLaunchKernelEx(&cfg, phs_linear_join_kernel, a, D * D / 4);
    cfg.numAttrs = 1;
  }
  if (err == cudaSuccess) {
    cfg.gridDim = dim3(a.B * a.Hkv * a.nseg * a.ngrp);
    cfg.blockDim = dim3(kLinThreads);
    cfg.dynamicSmemBytes = kRows;
    err = cudaLaunchKernelEx(&cfg, rows, tq, tk, tv, to, a);
  }
  if (err != cudaSuccess) return PHS_ECUDA;
  return cudaGetLastError() == cudaSuccess ? PHS_OK : PHS_ECUDA;
}

int launch_linear_prompt(int D, const CUtensorMap& tq, const CUtensorMap& tk,
                         const CUtensorMap& tv, const CUtensorMap& to, const LinearArgs& a,
                         cudaStream_t stream) {
  return D == 128 ? launch_linear_prompt_t<128>(tq, tk, tv, to, a, stream)
                  : launch_linear_prompt_t<64>(tq, tk, tv, to, a, stream);
}

}  // namespace phs
