// phs_write.cu -- rotary positions, tokens on their way into the paged cache
// (bf16 pages and 8-bit blocks), and the cache read back as rows.
//
// A position adds turns[i] / 2^64 of a full turn to pair i's angle.  position *
// turns[i] in 64-bit integers is exact modulo a turn, so a far position's
// angle is as good as a near one's; its top 32 bits go to sincospi.
#include "phs_common.cuh"
#include "phs_layers.h"
#include "phs_quant.cuh"

namespace phs {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float2 turn_cs(uint64_t turns, int pos, float factor) {
  const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(pos)) * turns;
  const int top = static_cast<int>(static_cast<uint32_t>(phase >> 32));
  float s, c;
  sincospif(static_cast<float>(top) * 0x1p-31f, &s, &c);
  return make_float2(c * factor, s * factor);
}

__device__ __forceinline__ float2 bf16_pair(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// A unit of a head's row is two 16-byte vectors: 8 pairs of elements where
// it is rotated (the first rotary / 16 units), else neighbours to copy.
__device__ __forceinline__ void unit_vecs(int u, int rotary, int interleaved, int& va, int& vb) {
  if (u < rotary / 16 && !interleaved) {
    va = u;
    vb = u + rotary / 16;
  } else {
    va = 2 * u;
    vb = 2 * u + 1;
  }
}

// The 8 pairs of a rotated unit by (cos, sin) pairs cs[0..7].
__device__ __forceinline__ void rotate_unit(uint4& va, uint4& vb, const float2* cs,
                                            int interleaved) {
  uint32_t* a = reinterpret_cast<uint32_t*>(&va);
  uint32_t* b = reinterpret_cast<uint32_t*>(&vb);
  if (interleaved) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 x = bf16_pair(a[e]), y = bf16_pair(b[e]), r = cs[e], t = cs[4 + e];
      a[e] = pack_bf16(fmaf(x.x, r.x, -(x.y * r.y)), fmaf(x.y, r.x, x.x * r.y));
      b[e] = pack_bf16(fmaf(y.x, t.x, -(y.y * t.y)), fmaf(y.y, t.x, y.x * t.y));
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 x = bf16_pair(a[e]), y = bf16_pair(b[e]), r = cs[2 * e], t = cs[2 * e + 1];
      a[e] = pack_bf16(fmaf(x.x, r.x, -(y.x * r.y)), fmaf(x.y, t.x, -(y.y * t.y)));
      b[e] = pack_bf16(fmaf(y.x, r.x, x.x * r.y), fmaf(y.y, t.x, x.y * t.y));
    }
  }
}

// Whether cu_seqlens is bad (decreases, or leaves [0, tokens]), one answer for
// the CTA; visit(b, lo, hi) gets each request's rows.  All threads call it.
template <class Visit>
__device__ __forceinline__ bool bad_ranges(const int32_t* cu, int B, int tokens, Visit&& visit) {
  int bad = 0;
  for (int j = threadIdx.x; j <= B; j += blockDim.x) {
    const int c = cu[j], next = j < B ? cu[j + 1] : c;
    bad |= c < 0 || c > tokens || next < c;
    if (j < B) visit(j, c, next);
  }
  return __syncthreads_or(bad);
}

// What a call does with request b.
struct Request {
  int n, len;    // new tokens, all tokens
  int qb, qa;    // tokens in 8 bits before and after
  bool ok, idle;
};
__device__ __forceinline__ Request request(const WriteArgs& a, int b) {
  Request r;
  r.n = a.cu_seqlens ? a.cu_seqlens[b + 1] - a.cu_seqlens[b] : 1;
  r.len = a.seq_lens[b];
  r.qb = r.qa = 0;
  r.idle = !a.cu_seqlens && r.len == 0;
  r.ok = !r.idle && r.len >= r.n;
  if (a.k_codes) {
    r.qb = a.qlens_before[b];
    r.qa = a.qlens[b];
    r.ok = r.ok && r.qb >= 0 && r.qb <= r.qa && r.qa <= r.len && (r.qb | r.qa) % kQBlock == 0 &&
           r.qb <= r.len - r.n && (r.qa - r.qb) / kQBlock <= a.max_qblocks;
  }
  return r;
}

// ------------------------------------------------------------ token rows --
// A CTA takes `tile` tokens: their requests, positions and pages once, the
// angles of their pairs once for all heads, then a thread one unit of a token
// over heads, four at a time with their loads in flight.  Each row is read
// and written once, so memory bounds it: 32,751 tokens of 32 query and 8 KV
// heads of 128 take 127 us, 120 for their bytes at the rate of a plain copy; a
// token of each of 256 requests 5 us of the GPU's time.
template <int D>
__global__ void __launch_bounds__(kThreads) phs_write_kernel(const __grid_constant__ WriteArgs a) {
  constexpr int U = D / 16;
  __shared__ int s_owner[kWriteMaxTile], s_pos[kWriteMaxTile], s_q[kWriteMaxTile];
  __shared__ int64_t s_row[kWriteMaxTile];  // row (head 0, token's slot) of its page, or -1
  __shared__ float2 s_cs[kWriteMaxTile][D / 2];
  // (from the last tokens on: beside 8-bit blocks these have the work, and the others'
  // CTAs end at once; 304 us against 317 for 65,521 tokens written and read back)
  const int tile = a.tile, r0 = (gridDim.x - 1 - blockIdx.x) * tile, r1 = min(r0 + tile, a.tokens);
  const int tid = threadIdx.x;
  bool refused = false;
  if (a.cu_seqlens) {
    if (tid < kWriteMaxTile) s_owner[tid] = -1;
    __syncthreads();
    refused = bad_ranges(a.cu_seqlens, a.B, a.tokens, [&](int b, int lo, int hi) {
      for (int r = max(lo, r0); r < min(hi, r1); ++r) s_owner[r - r0] = b;
    });
  }
  if (refused && tid == 0) set_status(a.status, PHS_ERANGE);
  if (tid < r1 - r0) {
    int pos = 0, q = 1;  // q: 1 rotated, 0 zero, -1 left alone
    int64_t row = -1;
    if (a.positions) {
      pos = a.positions[r0 + tid];
    } else {
      const int b = refused ? -1 : a.cu_seqlens ? s_owner[tid] : r0 + tid;
      if (b < 0) {
        q = -1;
      } else {
        const Request r = request(a, b);
        if (!r.ok) {
          q = 0;
          if (!r.idle) set_status(a.status, PHS_ERANGE);
        } else {
          pos = r.len - r.n + (a.cu_seqlens ? r0 + tid - a.cu_seqlens[b] : 0);
          if (pos < r.qa) {
            if (a.q_with_blocks) q = -1;
          } else {
            const int lp = pos / kPage;
            const int page =
                lp < a.max_pages ? a.block_table[static_cast<size_t>(b) * a.max_pages + lp] : -1;
            if (page < 0 || page >= a.num_pages)
              set_status(a.status, PHS_ERANGE);
            else if (a.page_refcount && a.page_refcount[page] != 1)
              set_status(a.status, PHS_ESHARED);
            else
              row = static_cast<int64_t>(page) * a.Hkv * kPage + pos % kPage;
          }
        }
      }
    }
    s_pos[tid] = pos;
    s_q[tid] = q;
    s_row[tid] = row;
  }
  if (!__syncthreads_or(tid < r1 - r0 && ((a.q && s_q[tid] >= 0) || a.k_out || s_row[tid] >= 0))) {
    pdl_wait_prior_grid();
    return;
  }
  const int half = a.rotary / 2;
  for (int e = tid; e < (r1 - r0) * half; e += kThreads)
    s_cs[e / half][e % half] = turn_cs(a.turns[e % half], s_pos[e / half], a.factor);
  __syncthreads();

  // queries and keys
  const int lanes = kThreads / (U * tile);  // heads at once
  const int u = tid % U, hl = tid / U % lanes, t = tid / U / lanes;
  int va, vb;
  unit_vecs(u, a.rotary, a.interleaved, va, vb);
  if (t < r1 - r0) {
    const int64_t row = s_row[t];
    const int q = a.q ? s_q[t] : -1, heads = a.Hq + (a.k ? a.Hkv : 0);
    const bool turned = u < a.rotary / 16;
    float2 cs[8];
    if (turned) {
#pragma unroll
      for (int e = 0; e < 8; ++e) cs[e] = s_cs[t][8 * u + e];
    }
    for (int h0 = hl; h0 < heads; h0 += 4 * lanes) {
      uint4 x[4], y[4];
      uint4* to[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int h = h0 + j * lanes;
        to[j] = nullptr;
        const uint4* from = nullptr;
        if (h < a.Hq) {
          if (q >= 0)
            to[j] = reinterpret_cast<uint4*>(a.q_out + (r0 + t) * a.q_out_stride + h * D);
          if (q > 0) from = reinterpret_cast<const uint4*>(a.q + (r0 + t) * a.q_stride + h * D);
        } else if (h < heads) {
          const int hk = h - a.Hq;
          if (a.k_out)
            to[j] = reinterpret_cast<uint4*>(a.k_out + (r0 + t) * a.k_out_stride + hk * D);
          else if (row >= 0)
            to[j] = reinterpret_cast<uint4*>(a.pool_k + (row + hk * kPage) * D);
          if (to[j]) from = reinterpret_cast<const uint4*>(a.k + (r0 + t) * a.k_stride + hk * D);
        }
        x[j] = y[j] = make_uint4(0, 0, 0, 0);
        if (from) {
          x[j] = from[va];
          y[j] = from[vb];
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (to[j]) {
          if (turned) rotate_unit(x[j], y[j], cs, a.interleaved);
          to[j][va] = x[j];
          to[j][vb] = y[j];
        }
    }
  }
  // values
  if (!a.v) return;
  constexpr int V = D / 8;
  const int per = a.Hkv * V;
  for (int e0 = tid; e0 < (r1 - r0) * per; e0 += 4 * kThreads) {
    uint4 x[4];
    uint4* to[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = e0 + j * kThreads, tt = e / per, c = e % per;
      to[j] = nullptr;
      if (tt < r1 - r0 && s_row[tt] >= 0) {
        x[j] = reinterpret_cast<const uint4*>(a.v + (r0 + tt) * a.v_stride)[c];
        to[j] = reinterpret_cast<uint4*>(a.pool_v + (s_row[tt] + c / V * kPage) * D) + c % V;
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (to[j]) *to[j] = x[j];
  }
  pdl_wait_prior_grid();  // (this grid's end must not come before that of the blocks' one)
}

// ---------------------------------------------------------- 8-bit blocks --
__device__ __forceinline__ uint32_t absmax16(const uint4& x, const uint4& y) {
  const uint32_t* a = reinterpret_cast<const uint32_t*>(&x);
  const uint32_t* b = reinterpret_cast<const uint32_t*>(&y);
  uint32_t m = 0u;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    asm("max.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(a[k]));
    asm("max.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(b[k]));
  }
  return m & 0x7FFF7FFFu;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// One CTA per (block of 32 tokens, some heads) of a request: a thread holds
// one unit of a token, K and V, head after head, and its pairs' angles for
// all of them.  A head's absmax meets in shared memory; V's codes are
// transposed there.  About 400 instructions a thread and head bound it (52 % of
// the issue slots, with the two barriers of a head): 65,521 tokens of 8 heads of
// 128 alone take 125 us, 60 for their bytes.  With `q_with_blocks` one more CTA
// a block turns the new tokens' queries, four heads in flight, which memory
// bounds: side by side both take 229 us for 32 query heads, 220 for their bytes.
// All 65,521 tokens written and read back, in a replayed graph: 304 us; with four
// CTAs an SM, and some spilled registers, 319; with three query heads in flight 311,
// with eight 370.  A warp for K or V of a head, with its 32 rows in registers and no
// barrier, has too few warps (a third slower).
template <int D>
__global__ void __launch_bounds__(2 * D, D == 128 ? 3 : 6)
    phs_write_block_kernel(const __grid_constant__ WriteArgs a, int heads_per_cta) {
  constexpr int U = D / 16, kWarps = D / 16;
  __shared__ uint32_t s_max[kWarps];
  __shared__ __align__(16) uint8_t s_v[kQBlock * D];  // V codes, token-major
  const int tid = threadIdx.x, b = blockIdx.y;
  const int groups = (a.Hkv + heads_per_cta - 1) / heads_per_cta;
  const int ctas = groups + a.q_with_blocks;  // of a block
  const int jr = blockIdx.x / ctas, h0 = blockIdx.x % ctas * heads_per_cta;
  const int h1 = min(h0 + heads_per_cta, a.Hkv);
  const bool queries = static_cast<int>(blockIdx.x % ctas) == groups;
  pdl_launch_dependents();
  bool refused = a.cu_seqlens &&
                 bad_ranges(a.cu_seqlens, a.B, a.tokens, [](int, int, int) {});
  Request r{};
  if (!refused) r = request(a, b);
  const bool say = tid == 0 && jr == 0 && h0 == 0;
  if (say && (refused || (!r.ok && !r.idle))) set_status(a.status, PHS_ERANGE);
  const int j = r.qb / kQBlock + jr;
  bool work = !refused && r.ok && j < r.qa / kQBlock;
  int qp = -1;
  if (work && !queries) {
    if (j < a.max_qpages) qp = a.qtable[static_cast<size_t>(b) * a.max_qpages + j];
    if (qp < 0 || qp >= a.num_qpages) {
      if (tid == 0) set_status(a.status, PHS_ERANGE);
      work = false;
    }
  }
  const int t = tid / U, u = tid % U, pos = j * kQBlock + t;
  const bool fresh = pos >= r.len - r.n;
  int va, vb;
  unit_vecs(u, a.rotary, a.interleaved, va, vb);
  const bool turned = fresh && u < a.rotary / 16;
  const uint4 *kp = nullptr, *vp = nullptr;
  int64_t step = D / 8;  // vectors from a head to the next
  float2 cs[8];
  if (queries) {
    if (!work || !fresh) return;
    if (turned) {
#pragma unroll
      for (int e = 0; e < 8; ++e) cs[e] = turn_cs(a.turns[8 * u + e], pos, a.factor);
    }
    const int64_t row = (a.cu_seqlens ? a.cu_seqlens[b] : b) + (pos - (r.len - r.n));
    const uint4* from = reinterpret_cast<const uint4*>(a.q + row * a.q_stride);
    uint4* to = reinterpret_cast<uint4*>(a.q_out + row * a.q_out_stride);
    constexpr int kAhead = 4;
#pragma unroll 1
    for (int h = 0; h < a.Hq; h += kAhead, from += kAhead * D / 8, to += kAhead * D / 8) {
      uint4 x[kAhead], y[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (h + i < a.Hq) {
          x[i] = from[i * D / 8 + va];
          y[i] = from[i * D / 8 + vb];
        }
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (h + i < a.Hq) {
          if (turned) rotate_unit(x[i], y[i], cs, a.interleaved);
          to[i * D / 8 + va] = x[i];
          to[i * D / 8 + vb] = y[i];
        }
    }
    return;
  }
  int bad = 0;
  if (work) {
    if (fresh) {
      const int64_t row = (a.cu_seqlens ? a.cu_seqlens[b] : b) + (pos - (r.len - r.n));
      kp = reinterpret_cast<const uint4*>(a.k + row * a.k_stride);
      vp = reinterpret_cast<const uint4*>(a.v + row * a.v_stride);
    } else {
      const int lp = pos / kPage;
      const int page =
          lp < a.max_pages ? a.block_table[static_cast<size_t>(b) * a.max_pages + lp] : -1;
      bad = page < 0 || page >= a.num_pages;
      if (!bad) {
        const int64_t at = (static_cast<int64_t>(page) * a.Hkv * kPage + pos % kPage) * (D / 8);
        kp = reinterpret_cast<const uint4*>(a.pool_k) + at;
        vp = reinterpret_cast<const uint4*>(a.pool_v) + at;
        step = kPage * D / 8;
      }
    }
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0) set_status(a.status, PHS_ERANGE);
    work = false;
  }
  if (!work) return;
  kp += h0 * step;
  vp += h0 * step;
  uint4 ka = kp[va], kb = kp[vb], xa = vp[2 * u], xb = vp[2 * u + 1];
  if (turned) {
#pragma unroll
    for (int e = 0; e < 8; ++e) cs[e] = turn_cs(a.turns[8 * u + e], pos, a.factor);
  }
  for (int h = h0; h < h1; ++h) {
    uint4 ka1 = ka, kb1 = kb, xa1 = xa, xb1 = xb;
    if (h + 1 < h1) {  // the next head's, while this one's absmax is found
      kp += step;
      vp += step;
      ka1 = kp[va];
      kb1 = kp[vb];
      xa1 = vp[2 * u];
      xb1 = vp[2 * u + 1];
    }
    if (turned) rotate_unit(ka, kb, cs, a.interleaved);
    const uint32_t mk = absmax16(ka, kb), mv = absmax16(xa, xb);
    // low half K, high half V
    uint32_t m = max2(__byte_perm(mk, mv, 0x5410), __byte_perm(mk, mv, 0x7632));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max2(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((tid & 31) == 0) s_max[tid >> 5] = m;
    __syncthreads();
    m = s_max[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) m = max2(m, s_max[w]);
    const float sk = __fdiv_rn(__uint_as_float(m << 16), 127.0f);
    const float sv = __fdiv_rn(__uint_as_float(m & 0xFFFF0000u), 127.0f);
    const float rk = sk != 0.f ? __fdiv_rn(1.0f, sk) : 0.f;
    const float rv = sv != 0.f ? __fdiv_rn(1.0f, sv) : 0.f;
    const uint64_t rk2 = f2(rk, rk), rv2 = f2(rv, rv);
    const size_t block = static_cast<size_t>(qp) * a.Hkv + h;
    uint2* ko = reinterpret_cast<uint2*>(a.k_codes + (block * kQBlock + t) * D);
    ko[va] = quant_codes8(reinterpret_cast<const uint32_t*>(&ka), sk, rk2, !(rk < INFINITY));
    ko[vb] = quant_codes8(reinterpret_cast<const uint32_t*>(&kb), sk, rk2, !(rk < INFINITY));
    const bool divide = !(rv < INFINITY);
    const uint2 c0 = quant_codes8(reinterpret_cast<const uint32_t*>(&xa), sv, rv2, divide);
    const uint2 c1 = quant_codes8(reinterpret_cast<const uint32_t*>(&xb), sv, rv2, divide);
    reinterpret_cast<uint4*>(s_v)[tid] = make_uint4(c0.x, c0.y, c1.x, c1.y);
    if (tid == 0) {
      a.k_scale[block] = sk;
      a.v_scale[block] = sv;
    }
    __syncthreads();
    // V^T: thread (half, word w of a row, q) transposes the 4 x 4 bytes of
    // words w of the four tokens of output word q; four threads then trade
    // words, so that each stores one dim's 16 bytes
    {
      constexpr int W = D / 4;
      const uint32_t* sw = reinterpret_cast<const uint32_t*>(s_v);
      const int q = tid & 3, w = tid / 4 % W, half = tid / (4 * W);
      const int t0 = 16 * half + 2 * q;  // tokens t0, t0 + 1, t0 + 8, t0 + 9: kI8VtToken
      const uint32_t r0 = sw[t0 * W + w], r1 = sw[(t0 + 1) * W + w];
      const uint32_t r2 = sw[(t0 + 8) * W + w], r3 = sw[(t0 + 9) * W + w];
      const uint32_t p0 = __byte_perm(r0, r1, 0x5140), p1 = __byte_perm(r0, r1, 0x7362);
      const uint32_t p2 = __byte_perm(r2, r3, 0x5140), p3 = __byte_perm(r2, r3, 0x7362);
      uint32_t o[4] = {__byte_perm(p0, p2, 0x5410), __byte_perm(p0, p2, 0x7632),
                       __byte_perm(p1, p3, 0x5410), __byte_perm(p1, p3, 0x7632)};
      // 4 x 4 transpose among the threads q: thread q gets dim 4 w + q
      const uint32_t e0 = __shfl_xor_sync(0xffffffffu, q & 1 ? o[0] : o[1], 1);
      const uint32_t e1 = __shfl_xor_sync(0xffffffffu, q & 1 ? o[2] : o[3], 1);
      if (q & 1) {
        o[0] = e0;
        o[2] = e1;
      } else {
        o[1] = e0;
        o[3] = e1;
      }
      const uint32_t e2 = __shfl_xor_sync(0xffffffffu, q & 2 ? o[0] : o[2], 2);
      const uint32_t e3 = __shfl_xor_sync(0xffffffffu, q & 2 ? o[1] : o[3], 2);
      if (q & 2) {
        o[0] = e2;
        o[1] = e3;
      } else {
        o[2] = e2;
        o[3] = e3;
      }
      reinterpret_cast<uint4*>(a.v_codes + block * kQBlock * D)[half * D + 4 * w + q] =
          make_uint4(o[0], o[1], o[2], o[3]);
    }
    ka = ka1;
    kb = kb1;
    xa = xa1;
    xb = xb1;
  }
}

// --------------------------------------------------------------- read back --
// One CTA per (page of 16 tokens, request).  65,521 tokens of 8 heads of 128, all but
// the last in 8 bits: 73 us, 60 for their bytes (91 with one load of K's codes in
// flight instead of four).
template <int D>
__global__ void __launch_bounds__(128) phs_read_back_kernel(const __grid_constant__ ReadArgs a) {
  constexpr int V = D / 8;
  const int b = blockIdx.y, tid = threadIdx.x;
  if (bad_ranges(a.cu_seqlens, a.B, a.tokens, [](int, int, int) {})) {
    if (tid == 0 && blockIdx.x == 0) set_status(a.status, PHS_ERANGE);
    return;
  }
  const int row0 = a.cu_seqlens[b], n = a.cu_seqlens[b + 1] - row0, start = a.starts[b];
  const int qlen = a.k_codes ? a.qlens[b] : 0;
  if (n > a.max_tokens || start < 0 || start > INT32_MAX - n - kPage || qlen < 0 ||
      qlen % kQBlock != 0) {
    if (tid == 0 && blockIdx.x == 0) set_status(a.status, PHS_ERANGE);
    return;
  }
  // (pages behind the request's last one end here: of a start near 2^31 their tokens
  // would pass it)
  if (n == 0 || static_cast<int>(blockIdx.x) > (start % kPage + n - 1) / kPage) return;
  const int lp = start / kPage + blockIdx.x, p0 = lp * kPage;
  const int lo = max(start, p0), hi = min(start + n, p0 + kPage);
  const bool codes = p0 < qlen;
  int page = -1;
  int64_t pages = codes ? a.num_qpages : a.num_pages;
  if (codes) {
    const int j = p0 / kQBlock;
    if (j < a.max_qpages) page = a.qtable[static_cast<size_t>(b) * a.max_qpages + j];
  } else if (lp < a.max_pages) {
    page = a.block_table[static_cast<size_t>(b) * a.max_pages + lp];
  }
  const bool missing = page < 0 || page >= pages;
  if (missing && tid == 0) set_status(a.status, PHS_ERANGE);
  const int count = hi - lo, first = lo - p0;
  const size_t per = static_cast<size_t>(a.Hkv) * V;  // vectors of an output row
  const size_t out0 = static_cast<size_t>(row0 + (lo - start)) * per;
  uint4* ko = reinterpret_cast<uint4*>(a.k_out) + out0;
  uint4* vo = reinterpret_cast<uint4*>(a.v_out) + out0;
  if (missing) {
    for (int e = tid; e < count * a.Hkv * V; e += 128) ko[e] = vo[e] = make_uint4(0, 0, 0, 0);
    return;
  }
  if (!codes) {
    const uint4* kp = reinterpret_cast<const uint4*>(a.pool_k) +
                      static_cast<size_t>(page) * a.Hkv * kPage * V;
    const uint4* vp = reinterpret_cast<const uint4*>(a.pool_v) +
                      static_cast<size_t>(page) * a.Hkv * kPage * V;
    const int cells = count * V;
    for (int e0 = tid; e0 < a.Hkv * cells; e0 += 4 * 128) {
      uint4 x[4], y[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = e0 + 128 * j, h = e / cells, c = e % cells;
        if (e < a.Hkv * cells) {
          x[j] = kp[(h * kPage + first) * V + c];
          y[j] = vp[(h * kPage + first) * V + c];
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = e0 + 128 * j, h = e / cells, c = e % cells;
        if (e < a.Hkv * cells) {
          const size_t to = (c / V) * per + h * V + c % V;
          ko[to] = x[j];
          vo[to] = y[j];
        }
      }
    }
    return;
  }
  // codes: byte x + 128 as the low byte of 2^23 + byte
  const auto value = [](uint32_t word, int byte, float scale) {
    return (__uint_as_float(__byte_perm(word, 0x4B000000u, 0x7440 | byte)) - 8388736.f) * scale;
  };
  const int half = p0 % kQBlock / kPage;
  const size_t block0 = static_cast<size_t>(page) * a.Hkv;
  const int cells = count * (V / 2);  // K: 16 codes of a token, four at once
  for (int e0 = tid; e0 < a.Hkv * cells; e0 += 4 * 128) {
    uint4 x[4];
    float s[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = e0 + 128 * j, h = e / cells, c = e % cells;
      if (e < a.Hkv * cells) {
        x[j] = reinterpret_cast<const uint4*>(
            a.k_codes + ((block0 + h) * kQBlock + 16 * half + first) * D)[c];
        s[j] = a.k_scale[block0 + h];
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = e0 + 128 * j, h = e / cells, c = e % cells, t = c / (V / 2), v = c % (V / 2);
      if (e >= a.Hkv * cells) break;
      const uint32_t* w = reinterpret_cast<const uint32_t*>(&x[j]);
      uint32_t y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        y[i] = pack_bf16(value(w[i / 2], 2 * (i & 1), s[j]),
                         value(w[i / 2], 2 * (i & 1) + 1, s[j]));
      uint4* to = ko + t * per + h * V + 2 * v;
      to[0] = make_uint4(y[0], y[1], y[2], y[3]);
      to[1] = make_uint4(y[4], y[5], y[6], y[7]);
    }
  }
  for (int e = tid; e < a.Hkv * V; e += 128) {  // V: 8 dims of the half's tokens
    const int h = e / V, v = e % V;
    const uint4* from = reinterpret_cast<const uint4*>(a.v_codes + (block0 + h) * kQBlock * D) +
                        half * D + 8 * v;
    uint4 x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = from[i];
    const float s = a.v_scale[block0 + h];
#pragma unroll
    for (int p = 0; p < 16; ++p) {
      const int t = kI8VtToken(p) - first;
      uint32_t y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        y[i] = pack_bf16(value(reinterpret_cast<const uint32_t*>(&x[2 * i])[p / 4], p & 3, s),
                         value(reinterpret_cast<const uint32_t*>(&x[2 * i + 1])[p / 4], p & 3, s));
      if (t >= 0 && t < count) vo[t * per + h * V + v] = make_uint4(y[0], y[1], y[2], y[3]);
    }
  }
}

template <int D>
int launch_write_t(WriteArgs a, int num_sms, cudaStream_t stream) {
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = stream;
  cfg.attrs = &early;
  const int64_t blocks = a.k_codes ? int64_t{a.max_qblocks} * a.B : 0;
  if (blocks > 0) {
    // The blocks' queries go with them where there are blocks enough to fill
    // the SMs: their copying then runs beside the blocks' arithmetic (304 us for
    // 65,521 tokens written and read back, 335 with the tokens' launch turning
    // them).  With fewer a CTA a block would turn its queries' heads one after
    // another, as it does where max_qblocks, a limit for every request, is
    // far above the blocks that there are (the host does not know their number).
    a.q_with_blocks = a.q && blocks >= int64_t{4} * num_sms;
    // All heads of a block by one CTA, which forms their angles once, unless
    // that leaves SMs without one; beside queries in halves, which end
    // together with those (304 us against 308; quarters 319).
    int per = a.q_with_blocks ? (a.Hkv + 1) / 2 : a.Hkv;
    while (per > 2 && blocks * ((a.Hkv + per - 1) / per) < int64_t{8} * num_sms)
      per = (per + 1) / 2;
    const int ctas = (a.Hkv + per - 1) / per + a.q_with_blocks;
    cfg.gridDim = dim3(a.max_qblocks * ctas, a.B);
    cfg.blockDim = dim3(2 * D);
    if (cudaLaunchKernelEx(&cfg, phs_write_block_kernel<D>, a, per) != cudaSuccess)
      return PHS_ECUDA;
    cfg.numAttrs = 1;  // the tokens start beside the blocks: they share no memory
  }
  if (a.tokens > 0) {
    cfg.gridDim = dim3((a.tokens + a.tile - 1) / a.tile);
    cfg.blockDim = dim3(kThreads);
    if (cudaLaunchKernelEx(&cfg, phs_write_kernel<D>, a) != cudaSuccess) return PHS_ECUDA;
  }
  return cudaGetLastError() == cudaSuccess ? PHS_OK : PHS_ECUDA;
}

}  // namespace

int launch_write(int D, WriteArgs a, int num_sms, cudaStream_t stream) {
  // Tiles as long as that leaves eight CTAs an SM (a limit of 1, 2 or 4: 45 to 49
  // us for 1,514 ragged tokens written and read back, within that call's own spread;
  // tiles of up to 8, 16 and 32 tokens: 312, 304 and 317 us for 65,521 tokens with
  // their queries by the blocks' launch, since more CTAs then have nothing to do).
  a.tile = kWriteMaxTile;
  while (a.tile > 1 && a.tokens < a.tile * 8 * num_sms) a.tile /= 2;
  return D == 128 ? launch_write_t<128>(a, num_sms, stream)
                  : launch_write_t<64>(a, num_sms, stream);
}

int launch_read_back(int D, const ReadArgs& a, cudaStream_t stream) {
  // a request's tokens may begin and end inside a page
  const dim3 grid((a.max_tokens + kPage - 2) / kPage + 1, a.B);
  if (D == 128)
    phs_read_back_kernel<128><<<grid, 128, 0, stream>>>(a);
  else
    phs_read_back_kernel<64><<<grid, 128, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? PHS_OK : PHS_ECUDA;
}

}  // namespace phs
