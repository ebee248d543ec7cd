// phs_scan_prompt.cu -- the selective scan over whole prompts.
//
// Prompts go in chunks of C = 128 tokens.  With l_t = s_t a a head's log decay
// in token t (s_t its step), L_i = sum_{t <= i} l_t within the chunk and S
// [P][N] the state before it, rows i, j of the chunk:
//   Y = diag(exp L_i) C S^T + (exp(L_i - L_j) s_j C B^T, j <= i) X + skip X
//   S <- exp(L_last) S + sum_j exp(L_last - L_j) s_j x_j b_j^T
// Four matrix products a chunk, on the tensor cores.  Heads of 64 go in pairs
// (a head of 128 as two halves), so that x, the state and the output are 128
// rows or columns ("slots" of 64, each with its head's decays):
//   QK = C B^T     128 x 128 x N    once for both slots
//   QS = C S^T     128 x 128 x N    A = C, B = S                (shared memory)
//   PV = P X       128 x 64 x 128   for each slot, A = P in tensor memory, B = X
//   KV = X'^T B    128 x N x 128    A = X'^T in tensor memory, B = B
// B, C and x are exact.  Decays make P (exp(L_i - L_j) s_j C B^T) a value of 24
// bits and the state is an fp32 one; both enter the rows' products as bf16, as
// their sums are rounded to bf16 in the end.  Each is off by up to 2^-8 of itself, a
// row by up to 2^-8 of its terms' absolute sum beside its own rounding; root mean
// square, and in units of that rounding's: 1.0 to 1.4 in all where b, c and x come
// out of a SiLU (1.03 to 1.08 with a skip of about 1), 1.1 to 1.5 where they are
// centred.  (Two terms of each, for 16 bits of them, leave that rounding alone; at
// the step that left them out 32,751 tokens of 64 heads took 509 us with them, 468
// without.)  The skip is added in fp32.
// What goes into the state keeps its 24 bits: X' (x times exp(L_last - L_j)
// s_j) enters as a sum of three bf16 terms, and KV is
// accumulated chunk by chunk from zero and added to the state in fp32 registers:
// the tensor cores' own sums drop the bits below the running sum's last one.
//
// A first small launch turns the steps into tables for each chunk and head.
// Sums of l that an exponential is taken of are formed over just their own
// tokens, never as differences of long sums (but within 32 tokens, for the
// blocks on the diagonal): exp(L_last - L_j) from sums from the end, the
// others by blocks of 32 tokens, exp(L_i - L_j) = exp(L_i - L_e) exp(L_e -
// L_j), e the last token of j's block.
//
// One CTA per (segment, pair of heads, request) walks its chunks in order:
//   warps 0-7   rows of the chunk, two threads a row: scores -> P, the
//               inter-chunk part scaled, the output rows
//   warps 8-15  rows of the state, two threads a row, in registers: state ->
//               shared memory, X tile -> X'^T terms (by warps 0-7 where only sums
//               are formed, which have no rows)
//   warp 16     issues KV
//   warp 17     TMA loads: a ring of B, C and X tiles
//   warp 18     TMA stores of the output tiles, in C's place
//   warp 19     issues QK, QS and PV
//
// Requests of a few tokens are left to a launch of their own (phs_scan.cu).
//
// Where there are fewer (request, pair) than SMs, prompts are cut into segments:
// a launch sums up their own states (B and X alone; a segment in `nsub` parts,
// as this launch has fewer CTAs), a small one joins these sums into the states
// that the segments start from, and the last one forms the rows.
//
// What bounds it: a chunk of a pair of heads (N = 128) takes some 9,500 cycles of a
// CTA, of which the tensor cores' products need 3,300 (their rates here: 32 cycles
// for a 128 x 64 x 16 product with A in tensor memory, 48 with both in shared
// memory, 62 for 128 wide ones) and the arithmetic of P, X' and the state about
// 2,800 of a scheduler.  The rest is the chain of steps through the roles, scores
// to P to PV to the rows and back to QS, with two or three warps a scheduler to
// hide each one's latency.  One prompt of 32,751 tokens, 64 heads of 64 and N =
// 128: 421 us (tables 14, sums of segments 90, join 8) against 101 for its bytes.
// What helped: P of both slots from one QK, in halves, so that PV and the next QK
// run beside the other half's P (577 -> 509); bf16 operands (-> 468); table values
// read a half ahead and only read there, since a warp waits where it computes
// with a load's result; loops instead of unrolled copies of P (-> 445); no copies
// to L2 ahead of the ring's (-> 421).  What did not: halves per slot with a QK
// each (548 -> 690, the tensor cores' time), a longer suspension in the waits (452
// -> 467), direct stores of the rows (467 -> 525), X ahead of C in the ring (425 ->
// 446), terms formed by all 16 warps of the sums' launch (421 -> 437), parts of X'
// ahead of the state: 0, 1, 2 of a warp 426, 421, 432.
#include "phs_prompt.cuh"
#include "phs_scan.cuh"

namespace phs {

namespace {

constexpr int kScanC = kScanChunk;
constexpr int kScanThreads = 640;
// registers a thread: 96 at launch, five warpgroups; 2 x 96 + 2 x 120 + 48 = 5 x 96
constexpr int kRegsRows = 96, kRegsState = 120, kRegsIssue = 48;
constexpr int kHalf = kScanC * 128;   // 64 columns of a tile: [128 rows][128 bytes]
constexpr int kTile = 2 * kHalf;      // a place of the ring

// A chunk's table of a head (floats).  Exponents of P in powers of two.
constexpr int kTabLoc = 0;      // sum of l from its 32 tokens' first one on
constexpr int kTabDiag = 128;   // the same less log2 s_j
constexpr int kTabCol = 256;    // exp(L_e - L_j) s_j, e the last of j's 32 tokens
constexpr int kTabEnd = 384;    // exp(L_last - L_j) s_j
constexpr int kTabFrom = 512;   // [4][4] of rows in block q for columns in block k <= q, at
                                // 4 k + q: what is added to kTabLoc for L_i - L_e, on the
                                // diagonal for L_i - L_m, or kNoRoom
constexpr int kTabBase = 528;   // [4] sum of l before each 32 tokens
constexpr int kTabTotal = 532;  // sum of l, natural
constexpr int kTabDecay = 533;  // its decay_factor
// On the diagonal exp(L_i - L_j) s_j is a product too, of exp(L_i - L_m) and exp(L_m -
// L_j) s_j, m the 16th of the 32 tokens, unless the first may be above 2^100 or the
// second leave 2^-124 to 2^124 (half of the 32 tokens decay by more, or steps are
// tiny or huge beside it): then each is taken by itself.
constexpr float kNoRoom = 1e30f;
static_assert(kScanTable == 536, "a table");

// Tensor-memory columns: a chunk's sum U, scores (and P), the outputs of both
// slots, and a ring of parts of X'^T (a step of 16 tokens: 3 terms of 8
// columns).
template <int N, bool STATES>
struct ScanTmem {
  static constexpr uint32_t kU = 0;
  static constexpr int kUBufs = STATES ? 2 : 1;
  static constexpr uint32_t kSc = 128, kOut = 256;
  static constexpr uint32_t kXp = STATES ? 256 : 384;
  static constexpr int kSteps = STATES ? 4 : 1;  // of 16 tokens
  static constexpr uint32_t kPart = 24 * kSteps;
  static constexpr int kRing = (512 - kXp) / kPart;
  static_assert(kXp + kRing * kPart <= 512, "tensor memory");
};

template <int N, bool STATES>
struct ScanLayout {
  static constexpr int kPer = STATES ? 2 : 3;  // tiles of a chunk: B, X (C between them)
  static constexpr int kSlots = 6;
  static constexpr int kS = kSlots * kTile;  // the state [N / 64][128 rows][128 bytes]
  static constexpr int kBar = STATES ? kS : kS + kScanC * N * 2;
  static constexpr int kBars = 2 * kSlots + 2 * ScanTmem<N, STATES>::kRing + 17;
  static constexpr int kMisc = kBar + kBars * 8;  // tensor-memory base, abort flag, request
  static constexpr int kCols = (kMisc + 16 + 15) / 16 * 16;  // a rows' warp: 2 rows of 32 floats
  static constexpr int kAlloc = kCols + (STATES ? 0 : 8 * 256);
  static_assert(kAlloc <= 227 * 1024, "shared memory of the prompt kernel");
};

// The n lowest bits (n >= 0).
__device__ __forceinline__ uint32_t low_bits(int n) {
  uint32_t r;
  asm("bmsk.clamp.b32 %0, 0, %1;" : "=r"(r) : "r"(n));
  return r;
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Row of the tables of request b's first chunk (t0 its first token): requests
// do not overlap, so neither do these.
__device__ __forceinline__ int64_t table_row(int b, int t0) { return t0 / kScanC + b; }

// The request that comes `at`-th when the longest come first (any short one where
// that one is short and another launch's).  Where there are more CTAs than SMs,
// the last ones to start then end soon.  All threads of the CTA call it.
__device__ __forceinline__ int scan_by_length(const ScanArgs& a, int at, volatile int* found) {
  static_assert(kScanSort <= kScanThreads, "a thread for each request");
  const int j = threadIdx.x;
  int64_t len = 0;
  if (j < a.B) len = int64_t{a.cu_seqlens[j + 1]} - a.cu_seqlens[j];
  const bool more = j < a.B && len > a.short_len;
  if (at >= __syncthreads_count(more)) {
    if (j < a.B && !more) *found = j;
  } else if (more) {
    int before = 0;
    int64_t from = a.cu_seqlens[0];
    for (int i = 0; i < a.B; ++i) {
      const int64_t to = a.cu_seqlens[i + 1];
      before += to - from > len || (to - from == len && i < j);
      from = to;
    }
    if (before == at) *found = j;
  }
  __syncthreads();
  return *found;
}

// ------------------------------------------------------------------ tables --
// One CTA per (chunk, request, 16 heads), a warp a head, a lane four tokens.
// A token's l is cut at -128: exp of that is zero in fp32, and sums that hold
// more would lose the bits of their neighbours.
constexpr int kTableHeads = 16;
__global__ void __launch_bounds__(32 * kTableHeads)
    phs_scan_table_kernel(const __grid_constant__ ScanArgs a) {
  __shared__ float s_step[kTableHeads][kScanC + 4];
  const int b = blockIdx.y, n = blockIdx.x, h0 = blockIdx.z * kTableHeads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, h = h0 + warp;
  pdl_launch_dependents();
  int t0, t1;
  if (!request_tokens(a, b, t0, t1) || t0 + n * kScanC >= t1 || t1 - t0 <= a.short_len) return;
  const int64_t row = table_row(b, t0) + n;
  t0 += n * kScanC;
  const int v = min(kScanC, t1 - t0);
  {  // two tokens of a warp at once
    const int k = lane & (kTableHeads - 1);
#pragma unroll
    for (int m = 0; m < kScanC / (2 * kTableHeads); ++m) {
      const int t = 2 * kTableHeads * m + 2 * warp + lane / kTableHeads;
      s_step[k][t] = t < v && h0 + k < a.H ? scan_step(a, t0 + t, h0 + k) : 0.f;
    }
  }
  __syncthreads();
  if (h >= a.H) return;
  constexpr float kLog2e = 1.4426950408889634f;
  const float rate = a.rate[h];
  const float4 s4 = *reinterpret_cast<const float4*>(&s_step[warp][4 * lane]);
  const float s[4] = {s4.x, s4.y, s4.z, s4.w};
  float l[4], own = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    l[e] = 4 * lane + e < v ? fmaxf(s[e] * rate, -128.f) : 0.f;
    own += l[e];
  }
  // sums of whole lanes: up to this one within its 8 (32 tokens), from it on
  // within its 8 and within all
  float pre = own, back32 = own, back = own;
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    const float x = __shfl_up_sync(0xffffffffu, pre, o, 8);
    if ((lane & 7) >= o) pre += x;
    const float y = __shfl_down_sync(0xffffffffu, back32, o, 8);
    if ((lane & 7) + o < 8) back32 += y;
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float x = __shfl_down_sync(0xffffffffu, back, o);
    if (lane + o < 32) back += x;
  }
  const float total = __shfl_sync(0xffffffffu, back, 0);
  const float block = __shfl_sync(0xffffffffu, pre, lane | 7);  // of these 32 tokens
  // the same without this lane's own tokens
  float after32 = __shfl_down_sync(0xffffffffu, back32, 1, 8);
  float after = __shfl_down_sync(0xffffffffu, back, 1);
  float before = __shfl_up_sync(0xffffffffu, pre, 1, 8);
  if ((lane & 7) == 7) after32 = 0.f;
  if (lane == 31) after = 0.f;
  if ((lane & 7) == 0) before = 0.f;
  float loc[4], diag[4], col[4], end[4], run = 0.f;
  float least = INFINITY, most = -INFINITY;  // log2 of the steps of these 32 tokens
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    run += l[e];
    loc[e] = (before + run) * kLog2e;
    const float log_s = log2f(s[e]);
    diag[e] = loc[e] - log_s;
    if (s[e] > 0.f) least = fminf(least, log_s);  // (a step of zero weighs nothing)
    most = fmaxf(most, log_s);
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    least = fminf(least, __shfl_xor_sync(0xffffffffu, least, o));
    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
  }
  const float first16 = __shfl_sync(0xffffffffu, loc[3], (lane & 24) + 3);
  run = 0.f;
#pragma unroll
  for (int e = 3; e >= 0; --e) {  // sums behind the token
    col[e] = ex2((after32 + run) * kLog2e) * s[e];
    end[e] = expf(after + run) * s[e];
    run += l[e];
  }
  float* tab = a.tables + (row * a.H + h) * kScanTable;
  reinterpret_cast<float4*>(tab + kTabLoc)[lane] = make_float4(loc[0], loc[1], loc[2], loc[3]);
  reinterpret_cast<float4*>(tab + kTabDiag)[lane] =
      make_float4(diag[0], diag[1], diag[2], diag[3]);
  reinterpret_cast<float4*>(tab + kTabCol)[lane] = make_float4(col[0], col[1], col[2], col[3]);
  reinterpret_cast<float4*>(tab + kTabEnd)[lane] = make_float4(end[0], end[1], end[2], end[3]);
  // blocks' sums, by every lane: x[q]
  float x[4], base = 0.f;
#pragma unroll
  for (int q = 0; q < 4; ++q) x[q] = __shfl_sync(0xffffffffu, block, 8 * q) * kLog2e;
  const float half16 = __shfl_sync(0xffffffffu, first16, 8 * (lane & 3));
  least = __shfl_sync(0xffffffffu, least, 8 * (lane & 3));
  most = __shfl_sync(0xffffffffu, most, 8 * (lane & 3));
  if (lane < 16) {  // lane 4 k + q
    const int k = lane >> 2, q = lane & 3;
    float from = 0.f;
    if (k == q) {
      const float rest = x[q] - half16;  // of the other 16
      const bool room = half16 > -100.f && rest > -100.f && half16 + least > -124.f &&
                        most - rest < 124.f;
      from = room ? -half16 : kNoRoom;
    }
#pragma unroll
    for (int m = 1; m < 3; ++m)
      if (k < m && m < q) from += x[m];
    tab[kTabFrom + lane] = from;
  }
#pragma unroll
  for (int q = 0; q < 3; ++q)
    if (q < lane) base += x[q];
  if (lane < 4) tab[kTabBase + lane] = base;
  if (lane == 0) {
    tab[kTabTotal] = total;
    tab[kTabDecay] = decay_factor(total);
  }
}

// -------------------------------------------------------------- the chunks --
// STATES: sums of each segment but the last, no outputs
template <int N, bool STATES>
__global__ void __launch_bounds__(kScanThreads, 1)
    phs_scan_prompt_kernel(const __grid_constant__ CUtensorMap tb,
                           const __grid_constant__ CUtensorMap tc,
                           const __grid_constant__ CUtensorMap tx,
                           const __grid_constant__ CUtensorMap to,
                           const __grid_constant__ ScanArgs a) {
  using L = ScanLayout<N, STATES>;
  using T = ScanTmem<N, STATES>;
  constexpr int kTermWarps = 2;  // that form X' of 32 columns of x
  constexpr int kTermThreads = 128 * kTermWarps;
  extern __shared__ __align__(1024) uint8_t smem[];  // (there is no other shared memory)
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // (known to be uniform)
  const int S = a.slots, rows = 64 * S;
  // part: the segment's first one, with STATES the one to sum up
  int b = blockIdx.x, unit = blockIdx.y, part = blockIdx.z;
  if (!STATES) {
    const int of_b = a.units * a.nseg, i = blockIdx.x % of_b;
    b = blockIdx.x / of_b;
    unit = i % a.units;
    part = i / a.units * a.nsub;
    if (a.longest_first)
      b = scan_by_length(a, b, reinterpret_cast<volatile int*>(smem + L::kMisc + 8));
  }
  const int col0 = unit * rows;                       // first column of x and of the output
  auto head = [&](int slot) { return (col0 + 64 * slot) / a.P; };
  const int group = head(0) / (a.H / a.G);

  // the join, or the short requests' launch, waits for this grid's end
  if (STATES || a.short_len >= 0) pdl_launch_dependents();

  // ---- this CTA's chunks
  const int64_t id = request_state(a, b);
  int t0, t1;
  if (!request_tokens(a, b, t0, t1) || t1 - t0 <= a.short_len) {
    pdl_wait_prior_grid();
    return;
  }
  const int all = (t1 - t0 + kScanC - 1) / kScanC, parts = a.nseg * a.nsub;
  const int next = part + (STATES ? 1 : a.nsub);
  const bool last = next == parts;
  const int c0 = part_chunk(a, all, part), c1 = part_chunk(a, all, next);
  if (c0 == c1 && !last) {
    pdl_wait_prior_grid();
    return;
  }
  // this CTA's first chunk's table of head 0
  const float* tables = a.tables + (table_row(b, t0) + c0) * a.H * kScanTable;
  t1 = min(t1, t0 + c1 * kScanC);
  t0 += c0 * kScanC;
  if (id < 0) {  // no state: zero rows
    if (!STATES)
      for (int64_t e = tid; e < static_cast<int64_t>(t1 - t0) * rows; e += kScanThreads)
        reinterpret_cast<__nv_bfloat16*>(a.out)[(t0 + e / rows) * a.H * a.P + col0 + e % rows] =
            __float2bfloat16_rn(0.f);
    pdl_wait_prior_grid();
    return;
  }
  const int nch = (t1 - t0 + kScanC - 1) / kScanC;
  const int head0 = head(0), head1 = head(S - 1);
  auto table = [&](int n, int slot) {
    return tables + (static_cast<int64_t>(n) * a.H + (slot ? head1 : head0)) * kScanTable;
  };

  // barriers: tile loaded / used, X' terms written / used; of a half of the
  // scores' columns: scores complete, P (and with the first half the
  // inter-chunk part) ready, P read; output tile written; state (the last
  // chunk's sum is read, the state written, rows behind the last token
  // zero), chunk sum complete; drain; inter-chunk part complete, outputs
  // complete, outputs read, all of the last chunk's KV issued
  auto bar = [sb](int i) { return sb + L::kBar + 8 * i; };
  constexpr int kB = 2 * L::kSlots, kR = kB + 2 * T::kRing;
  const uint32_t full = bar(0), empty = bar(L::kSlots), xp_full = bar(kB),
                 xp_empty = bar(kB + T::kRing), sc_full = bar(kR), pv_ready = bar(kR + 2),
                 pv_done = bar(kR + 4), y_full = bar(kR + 6), s_ready = bar(kR + 8),
                 u_done = bar(kR + 10), drain = bar(kR + 12), qs_done = bar(kR + 14),
                 o_free = bar(kR + 15), kv_all = bar(kR + 16);
  const uint32_t o_done = pv_done + 8;  // (PV of the second half is the last)
  static_assert(kR + 17 == L::kBars, "barriers (the first seven of these: pairs)");
  volatile int* abort = reinterpret_cast<volatile int*>(smem + L::kMisc + 4);
  if (warp == 16) {
    tmem_alloc(sb + L::kMisc, 512);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < L::kSlots; ++i) {
      mbar_init(full + 8 * i, 1);
      // whatever tile is in a place, two let go of it: of B QK and KV, of C QS
      // and the output's store, of X KV (whose terms have then been formed) and PV
      mbar_init(empty + 8 * i, STATES ? 1 : 2);
    }
    for (int i = 0; i < T::kRing; ++i) {
      mbar_init(xp_full + 8 * i, 128);
      mbar_init(xp_empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(sc_full + 8 * i, 1);
      mbar_init(pv_ready + 8 * i, 256);
      mbar_init(pv_done + 8 * i, 1);
      mbar_init(y_full + 8 * i, 256);
      mbar_init(drain + 8 * i, 1);
    }
    for (int i = 0; i < T::kUBufs; ++i) {
      mbar_init(s_ready + 8 * i, 256);
      mbar_init(u_done + 8 * i, STATES ? 1 : 2);  // KV, and QS done with the state
    }
    mbar_init(qs_done, 1);
    mbar_init(o_free, 256);
    mbar_init(kv_all, 1);
    *abort = 0;
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem =
      __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(smem + L::kMisc), 0);
  const uint32_t my_lanes = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
  // tile i of the ring: its place, its barriers, which turn of the place it is
  auto place_of = [sb](int i) { return sb + (i % L::kSlots) * kTile; };
  auto full_of = [&](int i) { return full + 8 * (i % L::kSlots); };
  auto empty_of = [&](int i) { return empty + 8 * (i % L::kSlots); };
  auto turn_of = [](int i) { return i / L::kSlots; };
  auto tile_b = [](int n) { return L::kPer * n; };
  auto tile_c = [](int n) { return L::kPer * n + 1; };
  auto tile_x = [](int n) { return L::kPer * n + L::kPer - 1; };

  constexpr int kBefore = STATES ? 0 : 1;  // parts of a warp before the state
  // parts of a chunk whose places in the ring are free when the state is there
  constexpr int kKnownFree = STATES ? 0 : T::kRing;

  // ---- X'^T of 32 columns of x, as three terms: ldmatrix.trans gives thread
  // 4 r + c tokens 2 c, 2 c + 1 (of 8) of column r of each of 4 groups of 8
  // columns.  The kTermWarps warps of these columns, of which this is number
  // `which`, take parts in turn.  `before(n)` is called ahead of the first.
  auto form_terms = [&](int which, auto&& before) {
    const int qt = warp & 3, kx = lane >> 3;  // matrix kx: columns 32 qt + 8 kx ..
    const bool mine = 32 * qt < rows;         // one slot: the upper half has no columns
    const uint32_t kcol = (qt >> 1) * kHalf + (lane & 7) * 128 +
                          ((((4 * (qt & 1) + kx) ^ lane) & 7) << 4);
    if (!mine && which == 0) {  // rows 64..127 of X'^T are zero
      uint32_t z[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) z[c] = 0u;
      for (uint32_t c = 0; c < T::kRing * T::kPart; c += 8)
#pragma unroll
        for (int x = 0; x < 2; ++x)
          tmem_st_16x128(my_lanes + (static_cast<uint32_t>(16 * x) << 16) + T::kXp + c, z);
      tmem_st_wait();
    }
    bool ok = true;
    int place = which, turn = 0;  // in the ring, of this warp's next part
    for (int n = 0; ok && n < nch; ++n) {
      const int v = min(kScanC, t1 - t0 - n * kScanC);
      const uint32_t xt = place_of(tile_x(n)), bt = place_of(tile_b(n));
      const float* weight = mine ? table(n, qt >> 1) + kTabEnd + 2 * (lane & 3) : nullptr;
      ok = lin_wait_warp(full_of(tile_x(n)), turn_of(tile_x(n)) & 1, abort);
      if (!ok) break;
      if (v < kScanC) {
        // rows behind the last token: no 0 * NaN.  X: what this warp reads
        // itself, its own parts' rows, since nothing orders it with the others
        // here; B: all (QK may read either; those scores are masked).
        ok = lin_wait_warp(full_of(tile_b(n)), turn_of(tile_b(n)) & 1, abort);
        if (!ok) break;
        for (int t = v + (lane >> 2); mine && t < kScanC; t += 8)
          if (t / (16 * T::kSteps) % kTermWarps == which)
            sts128(xt + (qt >> 1) * kHalf + t * 128 +
                       ((((4 * (qt & 1) + (lane & 3)) ^ t) & 7) << 4),
                   0, 0, 0, 0);
        for (int u = 128 * which + 32 * qt + lane; u < N / 64 * (kScanC - v) * 8;
             u += kTermThreads) {
          const int hf = u / ((kScanC - v) * 8), x = u % ((kScanC - v) * 8);
          sts128(bt + hf * kHalf + v * 128 + x * 16, 0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
      constexpr int kParts = kScanC / 16 / T::kSteps;
      // weights of a step's tokens, a step ahead
      float2 ahead[2];
      auto weights_of = [&](int t) {
        if (mine)
#pragma unroll
          for (int q = 0; q < 2; ++q)
            ahead[q] = *reinterpret_cast<const float2*>(weight + t + 8 * q);
      };
      weights_of(16 * T::kSteps * which);
#pragma unroll 1
      for (int p = which; ok && p < kParts + kTermWarps; p += kTermWarps) {
        if (p / kTermWarps == kBefore) ok = before(n);
        if (!ok || p >= kParts) break;
        // (a wait costs 100 cycles even where it has nothing to wait for: what
        // the last chunk had in the ring is known to be read once its sum is there)
        if (turn > 0 && (p / kTermWarps < kBefore || p >= kKnownFree))
          ok = lin_wait_warp(xp_empty + 8 * place, (turn - 1) & 1, abort);
        if (!ok) break;
        tc_fence_after();
        if (mine) {
#pragma unroll 1
          for (int st = 0; st < T::kSteps; ++st) {
            const int t = 16 * (T::kSteps * p + st);  // first token
            const float2 now[2] = {ahead[0], ahead[1]};
            const int t_next =
                st + 1 < T::kSteps ? t + 16 : t + 16 + 16 * T::kSteps * (kTermWarps - 1);
            if (t_next < kScanC) weights_of(t_next);
            uint32_t w[3][2][4];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              uint32_t k[4];
              ldsm_x4_t(xt + kcol + (t + 8 * q) * 128, k[0], k[1], k[2], k[3]);
              const uint64_t f = f2(now[q].x, now[q].y);
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
                tmem_st_16x128(my_lanes + (static_cast<uint32_t>(16 * x) << 16) + T::kXp +
                                   T::kPart * place + 24 * st + 8 * i,
                               w[i][x]);
          }
          tmem_st_wait();
        }
        tc_fence_before();
        mbar_arrive(xp_full + 8 * place);
        if ((place += kTermWarps) >= T::kRing) {
          place -= T::kRing;
          ++turn;
        }
      }
    }
    return ok;
  };

  // The first tiles are on their way while an earlier launch ends; all else
  // waits for that end here, not in a wait of limited length.
  if (warp != 17) pdl_wait_prior_grid();

  // (each warpgroup sets its registers at the head of its own branch, so that
  // the code behind it is compiled for that number)
  if (warp >= 16) {
    regs_dec<kRegsIssue>();
    if (warp == 17) {
      // ---------------------------------------------------------------- TMA
      if (lane == 0 && nch > 0) {
        prefetch_tmap(&tb);
        prefetch_tmap(&tx);
        if (!STATES) prefetch_tmap(&tc);
        const uint64_t pol = policy_evict_first();
        bool ok = true;
        int tiles = 0;
        auto load = [&](const CUtensorMap* map, int col, int halves, int t) {
          if (turn_of(tiles) > 0)
            ok = ok && lin_wait(empty_of(tiles), (turn_of(tiles) - 1) & 1, abort);
          if (!ok) return;
          mbar_arrive_expect_tx(full_of(tiles), halves * kHalf);
          for (int hf = 0; hf < halves; ++hf)
            tma_load_2d(place_of(tiles) + hf * kHalf, map, col + 64 * hf, t, full_of(tiles), pol);
          ++tiles;
        };
        for (int n = 0; ok && n < nch; ++n) {
          const int t = t0 + n * kScanC;
          load(&tb, group * N, N / 64, t);
          if (!STATES && ok) load(&tc, group * N, N / 64, t);
          if (ok) load(&tx, col0, S, t);
          if (n == 0) pdl_wait_prior_grid();
        }
        if (!ok) {
          set_status(a.status, PHS_ETIMEOUT);
          *abort = 1;
        }
        // copies still in flight land before the CTA ends
        for (int i = max(0, tiles - L::kSlots); i < tiles; ++i)
          (void)mbar_wait(full_of(i), turn_of(i) & 1);
      }
    } else if (warp == 16 || (!STATES && warp == 19)) {
      // ----------------------------------------------------------- products
      // (a whole warp walks the chunks and one elected lane issues, so that the
      // compiler keeps what the instructions take in uniform registers)
      constexpr uint32_t kIdQK = idesc_bf16_f32(128, 64, false, false);
      const uint32_t id_qs = S == 2 ? idesc_bf16_f32(128, 128, false, false) : kIdQK;
      constexpr uint32_t kIdKV = idesc_bf16_f32(128, N, false, true);
      constexpr uint32_t kIdPV = idesc_bf16_f32(128, 64, false, true);
      bool ok = true;
      const bool lead = elect_one();
      auto wait = [&](uint32_t bar, int turn) {
        ok = ok && lin_wait_warp(bar, turn & 1, abort);
      };
      auto tile_full = [&](int i) { wait(full_of(i), turn_of(i)); };
      if (warp == 16) {  // KV
        int place = 0, turn = 0;  // of the next part of X'
        for (int n = 0; ok && n < nch; ++n) {
          const int ub = n % T::kUBufs;
          tile_full(tile_b(n));
          tile_full(tile_x(n));
          if (!STATES)
            wait(s_ready, n);
          else if (n >= 2)  // the sum two chunks ago has been taken up
            wait(s_ready + 8 * ub, n / 2 - 1);
          uint64_t v = sdesc_sw128(place_of(tile_b(n)), kHalf, 1024);
#pragma unroll 1
          for (int p = 0; p < kScanC / 16; p += T::kSteps, v += T::kSteps * 2048 >> 4) {
            wait(xp_full + 8 * place, turn);
            if (!ok) break;
            tc_fence_after();
            if (lead) {
              const uint32_t xp = tmem + T::kXp + T::kPart * place;
#pragma unroll
              for (int t = 0; t < 3; ++t)
#pragma unroll
                for (int st = 0; st < T::kSteps; ++st)
                  umma_bf16_ts(tmem + T::kU + N * ub, xp + 24 * st + 8 * t, v + (st * 2048 >> 4),
                               kIdKV, p > 0 || t > 0 || st > 0);
              umma_commit(xp_empty + 8 * place);
            }
            __syncwarp();
            if (++place == T::kRing) {
              place = 0;
              ++turn;
            }
          }
          if (ok && lead) {
            // (PV of a chunk with rows behind the last token waits for their zeros)
            if (!STATES && t1 - t0 < (n + 1) * kScanC) mbar_arrive(kv_all);
            umma_commit(u_done + 8 * ub);
            umma_commit(empty_of(tile_b(n)));
            umma_commit(empty_of(tile_x(n)));
          }
          __syncwarp();
        }
      } else {  // QK, QS, PV
        // By halves of the scores' columns: while the rows' warps form P of one,
        // the other's PV and the next chunk's QK run.
        const uint64_t ds = sdesc_sw128(sb + L::kS, 16, 1024);
        auto issue_qk = [&](int n, int hh) {
          if (hh == 0) {
            tile_full(tile_b(n));
            tile_full(tile_c(n));
          }
          if (!ok) return;
          tc_fence_after();
          const uint64_t db = sdesc_sw128(place_of(tile_b(n)) + hh * (kHalf / 2), 16, 1024);
          const uint64_t dc = sdesc_sw128(place_of(tile_c(n)), 16, 1024);
          if (lead) {
#pragma unroll 4
            for (int ks = 0; ks < N / 16; ++ks) {
              const uint32_t at = ((ks >> 2) * kHalf + (ks & 3) * 32) >> 4;
              umma_bf16(tmem + T::kSc + 64 * hh, dc + at, db + at, kIdQK, ks > 0);
            }
            umma_commit(sc_full + 8 * hh);
            if (hh == 1) umma_commit(empty_of(tile_b(n)));
          }
          __syncwarp();
        };
        if (nch > 0) {
          issue_qk(0, 0);
          if (ok) issue_qk(0, 1);
        }
        for (int n = 0; ok && n < nch; ++n) {
          wait(s_ready, n);
          if (n > 0) wait(o_free, n - 1);
          if (!ok) break;
          tc_fence_after();
          const uint64_t dc = sdesc_sw128(place_of(tile_c(n)), 16, 1024);
          if (lead) {
#pragma unroll 4
            for (int ks = 0; ks < N / 16; ++ks) {
              const uint32_t at = ((ks >> 2) * kHalf + (ks & 3) * 32) >> 4;
              umma_bf16(tmem + T::kOut, dc + at, ds + at, id_qs, ks > 0);
            }
            umma_commit(qs_done);
            umma_commit(u_done);  // the state has been read
            umma_commit(empty_of(tile_c(n)));
          }
          __syncwarp();
          tile_full(tile_x(n));
          if (t1 - t0 < (n + 1) * kScanC) wait(kv_all, 0);
          for (int hh = 0; ok && hh < 2; ++hh) {
            wait(pv_ready + 8 * hh, n);
            if (!ok) break;
            tc_fence_after();
            const uint64_t v = sdesc_sw128(place_of(tile_x(n)) + hh * (kHalf / 2), kHalf, 1024);
            if (lead) {
#pragma unroll 1
              for (int s = 0; s < S; ++s)
#pragma unroll
                for (int ks = 0; ks < kScanC / 32; ++ks)
                  umma_bf16_ts(tmem + T::kOut + 64 * s,
                               tmem + T::kSc + 64 * hh + 16 * ks + 8 * s,
                               v + ((s * kHalf + ks * 2048) >> 4), kIdPV, 1u);
              umma_commit(pv_done + 8 * hh);
              if (hh == 1) umma_commit(empty_of(tile_x(n)));
            }
            __syncwarp();
            wait(pv_done + 8 * hh, n);  // P is read
            if (ok && n + 1 < nch) issue_qk(n + 1, hh);
          }
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
        const int whole = (t1 - t0) / kScanC;  // (the others' rows are stored by the threads)
        bool ok = true;
        for (int n = 0; ok && n < nch; ++n) {
          ok = lin_wait(y_full + 8 * (n & 1), (n >> 1) & 1, abort);
          if (!ok) break;
          if (n < whole) {
            for (int hf = 0; hf < S; ++hf)
              tma_store_2d(&to, place_of(tile_c(n)) + hf * kHalf, col0 + 64 * hf,
                           t0 + n * kScanC);
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
          }
          mbar_arrive(empty_of(tile_c(n)));
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
    regs_dec<kRegsRows>();
    const int qt = warp & 3, half = warp >> 2, i = 32 * qt + lane;  // row
    bool ok = true;
    // What a slot takes from its table for a half of the columns: this row's L
    // from its 32 tokens' first one on, what to add to it, the column `lane`s
    // factor, L before the 32 tokens.  Read ahead, and only read there: the
    // warp would wait where it computes with them.
    struct Ahead {
      float loc, from, col, base;
    } next[2] = {};
    auto read_ahead = [&](int n, int hh) {
      if (n >= nch) return;
      const int kb = 2 * hh + half;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (s >= S) break;
        const float* tab = table(n, s);
        next[s].loc = tab[kTabLoc + i];
        next[s].base = tab[kTabBase + qt];
        if (kb <= qt) {
          next[s].from = tab[kTabFrom + 4 * kb + qt];
          next[s].col = tab[(kb < qt ? kTabCol : kTabDiag) + 32 * kb + lane];
        }
      }
    };
    const float skip0 = a.skip ? a.skip[head0] : 0.f, skip1 = a.skip ? a.skip[head1] : 0.f;
    float* const cols = reinterpret_cast<float*>(smem + L::kCols + 256 * warp);
    // P of a half of the columns in place of the scores: 32 columns a thread,
    // block kb of 32 tokens; 16 columns of a step of the product become 8 of
    // each slot
    auto form_p = [&](int n, int hh) {
      const int kb = 2 * hh + half;
      const uint32_t at = my_lanes + T::kSc + 32 * kb;
      const bool whole = kb < qt || (next[0].from < kNoRoom && next[1].from < kNoRoom);
      float c0 = next[0].col, c1 = next[1].col;
      if (kb == qt && whole) {
        c0 = ex2(-next[0].from - c0);
        c1 = ex2(-next[1].from - c1);
      }
      __syncwarp();  // (the last half's columns have been read)
      cols[lane] = c0;
      cols[32 + lane] = c1;
      __syncwarp();
      const float f0 = ex2(next[0].loc + next[0].from), f1 = ex2(next[1].loc + next[1].from);
      ok = lin_wait_warp(sc_full + 8 * hh, n & 1, abort);
      if (!ok) return;
      tc_fence_after();
      if (kb > qt) {  // behind every row
        uint32_t p[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) p[e] = 0u;
        tmem_st16(at, p);
        tmem_st16(at + 16, p);
        return;
      }
#pragma unroll 1
      for (int k = 0; k < 2; ++k) {
        uint32_t sc[16];
        tmem_ld16(at + 16 * k, sc);
        tmem_ld_wait();
        const int d = lane - 16 * k;  // column of the diagonal
#pragma unroll 1
        for (int s = 0; s < S; ++s) {
          const float4* c4 = reinterpret_cast<const float4*>(cols + 32 * s + 16 * k);
          const uint64_t f = s ? f2(f1, f1) : f2(f0, f0);
          uint32_t p[8];
          if (kb < qt) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float4 c = c4[e];
              const uint32_t* x = sc + 4 * e;
              p[2 * e] = pack_term(f2_mul(f2(x[0], x[1]), f2_mul(f, f2(c.x, c.y))));
              p[2 * e + 1] = pack_term(f2_mul(f2(x[2], x[3]), f2_mul(f, f2(c.z, c.w))));
            }
          } else {
            const float row = s ? next[1].loc : next[0].loc;
            uint64_t w[8];
            if (whole) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float4 c = c4[e];
                w[2 * e] = f2_mul(f, f2(c.x, c.y));
                w[2 * e + 1] = f2_mul(f, f2(c.z, c.w));
              }
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float4 c = c4[e];
                w[2 * e] = f2(ex2(row - c.x), ex2(row - c.y));
                w[2 * e + 1] = f2(ex2(row - c.z), ex2(row - c.w));
              }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const bool in0 = d >= 2 * e, in1 = d >= 2 * e + 1;
              const float2 x = f2_get(f2_mul(f2(sc[2 * e], sc[2 * e + 1]), w[e]));
              p[e] = pack_bf16(in0 ? x.x : 0.f, in1 ? x.y : 0.f);
            }
          }
          tmem_st8(at + 16 * k + 8 * s, p);
        }
      }
    };
    read_ahead(0, 0);
#pragma unroll 1
    for (int n = 0; ok && n < nch; ++n) {
#pragma unroll 1
      for (int hh = 0; hh < 2; ++hh) {
        form_p(n, hh);
        if (!ok) break;
        if (hh == 0) {  // the part before the chunk scaled in place, and the skip
          ok = lin_wait_warp(qs_done, n & 1, abort);
          if (!ok) break;
          tc_fence_after();
          const float g0 = ex2(next[0].loc + next[0].base), g1 = ex2(next[1].loc + next[1].base);
          read_ahead(n, 1);
          ok = lin_wait_warp(full_of(tile_x(n)), turn_of(tile_x(n)) & 1, abort);
          if (!ok) break;
          const uint32_t xrow = place_of(tile_x(n)) + i * 128;
#pragma unroll 1
          for (int s = 0; s < S; ++s) {
            const uint64_t f = s ? f2(g1, g1) : f2(g0, g0);
            const float skip = s ? skip1 : skip0;
            uint32_t o[32];
            const uint32_t at = my_lanes + T::kOut + 64 * s + 32 * half;
            tmem_ld32(at, o);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint4 x = lds128(xrow + s * kHalf + ((((4 * half + k) ^ i) & 7) << 4));
              const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int m = 0; m < 4; ++m) {
                const int e = 8 * k + 2 * m;
                const float2 y = f2_get(
                    f2_fma(f2(o[e], o[e + 1]), f,
                           f2_mul(f2(w[m] << 16, w[m] & 0xFFFF0000u), f2(skip, skip))));
                o[e] = __float_as_uint(y.x);
                o[e + 1] = __float_as_uint(y.y);
              }
            }
            tmem_st32(at, o);
          }
        } else {
          read_ahead(n + 1, 0);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(pv_ready + 8 * hh);
      }
      // output rows: a whole chunk's go through shared memory (in place of C,
      // whose products are complete) and TMA; the rows behind a last token are
      // another request's
      ok = ok && lin_wait_warp(o_done, n & 1, abort);
      if (!ok) break;
      tc_fence_after();
      const int t = t0 + n * kScanC + i;
      const bool whole = t0 + (n + 1) * kScanC <= t1;
      const uint32_t row = place_of(tile_c(n)) + i * 128;
      uint4* to_row = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.out) +
                                               static_cast<size_t>(t) * a.H * a.P + col0);
#pragma unroll 1
      for (int s = 0; s < S; ++s) {
        uint32_t o[32];
        tmem_ld32(my_lanes + T::kOut + 64 * s + 32 * half, o);
        tmem_ld_wait();
        uint4 y[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float* x = reinterpret_cast<const float*>(o + 8 * k);
          y[k] = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                            pack_bf16(x[6], x[7]));
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int u = 4 * half + k;  // 16 bytes of the slot's row
          if (whole)
            sts128(row + s * kHalf + (((u ^ i) & 7) << 4), y[k].x, y[k].y, y[k].z, y[k].w);
          else if (t < t1)
            to_row[8 * s + u] = y[k];
        }
      }
      tc_fence_before();
      mbar_arrive(o_free);
      if (whole) fence_proxy_async_smem();
      mbar_arrive(y_full + 8 * (n & 1));
    }
    if (!ok) {
      set_status(a.status, PHS_ETIMEOUT);
      *abort = 1;
    }
  } else if (STATES && warp < 8) {
    regs_dec<kRegsRows>();
    if (!form_terms(warp >> 2, [](int) { return true; })) {
      set_status(a.status, PHS_ETIMEOUT);
      *abort = 1;
    }
  } else {
    // ------------------------------------------------- rows of the state
    regs_inc<kRegsState>();
    constexpr int M = N / 2;  // columns of a thread
    const int qt = warp & 3, half = (warp >> 2) & 1;
    const int r = 32 * qt + lane;  // row; one slot: the upper half has none
    const bool mine = r < rows;
    const size_t row = static_cast<size_t>(r) * N + half * M;
    float* pool = a.state + (id * a.H * a.P + col0) * N + row;
    const size_t sums = static_cast<size_t>(b) * a.units + unit;  // of the parts' sums
    float* ws = a.ws + (sums * parts + part) * rows * N + row;
    const bool resume = a.resume != nullptr && a.resume[b] != 0;
    uint64_t R[M / 2];  // pairs
#pragma unroll
    for (int c = 0; c < M / 2; ++c) R[c] = 0ull;
    if (mine && !STATES && (part > 0 || resume)) {
      const float* from = a.nseg > 1 ? ws : pool;
#pragma unroll
      for (int c = 0; c < M; c += 4) {
        const float4 x = *reinterpret_cast<const float4*>(from + c);
        R[c / 2] = f2(x.x, x.y);
        R[c / 2 + 1] = f2(x.z, x.w);
      }
    }
    bool ok = true;
    float log = 0.f;                           // of the part's decay
    float decay = mine && nch > 0 ? table(0, qt >> 1)[kTabDecay] : 0.f;  // a chunk ahead
    float total = STATES && mine && nch > 0 ? table(0, qt >> 1)[kTabTotal] : 0.f;
    // R <- state after chunk n (n >= 0), and where `store` as bf16 to shared
    // memory for the next chunk's QS (u_done counts the last one's reads too)
    auto next_state = [&](int n, bool store) {
      const int ub = n >= 0 ? n % T::kUBufs : 0;
      uint64_t factor = 0ull, base = 0ull;
      if (n >= 0 && mine) {
        const float d = decay, one = is_small_decay(d) ? 1.f : 0.f;
        if (STATES) log += total;
        if (n + 1 < nch) decay = table(n + 1, qt >> 1)[kTabDecay];
        if (STATES && n + 1 < nch) total = table(n + 1, qt >> 1)[kTabTotal];
        factor = f2(d, d);
        base = f2(one, one);
      }
      if (n >= 0) {
        ok = ok && lin_wait_warp(u_done + 8 * ub, n / T::kUBufs & 1, abort);
        if (!ok) return;
        tc_fence_after();
      }
      if (mine) {
        const uint32_t my_row = sb + L::kS + r * 128;
#pragma unroll
        for (int c = 0; c < M / 16; ++c) {
          if (n >= 0) {
            uint32_t u[16];
            tmem_ld16(my_lanes + T::kU + N * ub + half * M + 16 * c, u);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 8; ++e)
              R[8 * c + e] = f2_add(f2_fma(R[8 * c + e], factor, f2_mul(R[8 * c + e], base)),
                                    f2(u[2 * e], u[2 * e + 1]));
          }
          if (store) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint64_t* x = R + 8 * c + 4 * k;
              const int u = half * (M / 8) + 2 * c + k;  // 16 bytes of the row
              sts128(my_row + (u >> 3) * kHalf + (((u ^ r) & 7) << 4), pack_term(x[0]),
                     pack_term(x[1]), pack_term(x[2]), pack_term(x[3]));
            }
          }
        }
        if (store) fence_proxy_async_smem();
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
      if (ok && nch > 0) next_state(nch - 1, false);
    }
    if (!ok) {
      set_status(a.status, PHS_ETIMEOUT);
      *abort = 1;
    } else if (mine && (STATES || last)) {
      float* at = STATES ? ws : pool;
#pragma unroll
      for (int c = 0; c < M; c += 4) {
        const float2 x = f2_get(R[c / 2]), y = f2_get(R[c / 2 + 1]);
        *reinterpret_cast<float4*>(at + c) = make_float4(x.x, x.y, y.x, y.y);
      }
      if (STATES && half == 0 && (r & 63) == 0)
        a.ws_log[(sums * parts + part) * 2 + (r >> 6)] = log;
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
// loads at once.
__global__ void __launch_bounds__(128) phs_scan_join_kernel(const __grid_constant__ ScanArgs a,
                                                            int N) {
  const int b = blockIdx.x, unit = blockIdx.y, rows = 64 * a.slots;
  const int vecs = rows * N / 4, i = blockIdx.z * 128 + threadIdx.x;
  pdl_launch_dependents();
  const int64_t id = request_state(a, b);
  int t0, t1;
  const bool good = request_tokens(a, b, t0, t1) && id >= 0 && t1 - t0 > a.short_len;
  pdl_wait_prior_grid();
  if (!good) return;
  const int chunks = (t1 - t0 + kScanC - 1) / kScanC, parts = a.nseg * a.nsub;
  const size_t first = (static_cast<size_t>(b) * a.units + unit) * parts;
  const float* log = a.ws_log + first * 2 + 4 * i / N / 64;  // this row's slot
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (a.resume && a.resume[b] != 0)
    s = reinterpret_cast<const float4*>(a.state + (id * a.H * a.P + unit * rows) * N)[i];
  float4* at = reinterpret_cast<float4*>(a.ws) + first * vecs + i;
  const int sums = parts - a.nsub;  // the last segment has none
  for (int n = 0; n <= sums; n += 8) {
    float4 x[8];
    float x_log[8];
    bool sum[8];  // not empty
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      sum[j] = n + j < sums && part_chunk(a, chunks, n + j) < part_chunk(a, chunks, n + j + 1);
      if (sum[j]) {
        x[j] = at[static_cast<size_t>(n + j) * vecs];
        x_log[j] = log[2 * (n + j)];
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (n + j <= sums && (n + j) % a.nsub == 0) at[static_cast<size_t>(n + j) * vecs] = s;
      if (sum[j]) {
        const float k = decay_factor(x_log[j]);
        s = make_float4(decayed(s.x, k) + x[j].x, decayed(s.y, k) + x[j].y,
                        decayed(s.z, k) + x[j].z, decayed(s.w, k) + x[j].w);
      }
    }
  }
}

template <int N>
int launch_scan_prompt_t(const CUtensorMap& tb, const CUtensorMap& tc, const CUtensorMap& tx,
                         const CUtensorMap& to, const ScanArgs& a, cudaStream_t stream) {
  constexpr int kStates = ScanLayout<N, true>::kAlloc, kRows = ScanLayout<N, false>::kAlloc;
  auto states = phs_scan_prompt_kernel<N, true>;
  auto rows = phs_scan_prompt_kernel<N, false>;
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
  cfg.gridDim = dim3(a.max_chunks, a.B, (a.H + kTableHeads - 1) / kTableHeads);
  cfg.blockDim = dim3(32 * kTableHeads);
  cudaError_t err = cudaLaunchKernelEx(&cfg, phs_scan_table_kernel, a);
  cfg.numAttrs = 1;
  if (err == cudaSuccess && a.nseg > 1) {
    cfg.gridDim = dim3(a.B, a.units, (a.nseg - 1) * a.nsub);
    cfg.blockDim = dim3(kScanThreads);
    cfg.dynamicSmemBytes = kStates;
    err = cudaLaunchKernelEx(&cfg, states, tb, tc, tx, to, a);
    if (err == cudaSuccess) {
      cfg.gridDim = dim3(a.B, a.units, 64 * a.slots * N / 512);
      cfg.blockDim = dim3(128);
      cfg.dynamicSmemBytes = 0;
      err = cudaLaunchKernelEx(&cfg, phs_scan_join_kernel, a, N);
    }
  }
  if (err == cudaSuccess) {
    cfg.gridDim = dim3(a.B * a.units * a.nseg);
    cfg.blockDim = dim3(kScanThreads);
    cfg.dynamicSmemBytes = kRows;
    err = cudaLaunchKernelEx(&cfg, rows, tb, tc, tx, to, a);
  }
  if (err == cudaSuccess && a.short_len >= 0) return launch_scan_short(a.P, N, a, true, stream);
  if (err != cudaSuccess) return PHS_ECUDA;
  return cudaGetLastError() == cudaSuccess ? PHS_OK : PHS_ECUDA;
}

}  // namespace

int launch_scan_prompt(int N, const CUtensorMap& tb, const CUtensorMap& tc, const CUtensorMap& tx,
                       const CUtensorMap& to, const ScanArgs& a, cudaStream_t stream) {
  return N == 128 ? launch_scan_prompt_t<128>(tb, tc, tx, to, a, stream)
                  : launch_scan_prompt_t<64>(tb, tc, tx, to, a, stream);
}

}  // namespace phs
