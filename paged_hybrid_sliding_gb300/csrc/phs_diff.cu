// phs_diff.cu -- differential attention of one new token per request over
// the paged pool.
//
//   out_i = (softmax(s q_{2i} K1) - lambda softmax(s q_{2i+1} K2)) V
//   lambda = exp(lambda_q1 . lambda_k1) - exp(lambda_q2 . lambda_k2) + lambda_init
// and, with a norm weight g,
//   out_i <- (1 - lambda_init) g out_i / sqrt(mean(out_i^2) + eps).
// Value head j of head i (j = i / (H / Hv)) has the two keys in pool heads
// 2j and 2j + 1 of K, and its 2D value columns in the same two heads of V.
//
// The step reads every K and V byte of the batch and computes 2 (D + 2D)
// multiply-adds per head and token, far below what the tensor cores do in
// that time: it is bound by the read.  Up to 8 heads of a value head share one
// read; 9 to 16 take two CTAs that each read it, the second mostly from L2 (16
// requests of 8,192 tokens, 16 heads on each of 4 value heads: 1.05 times the
// bytes from HBM, but 148 us against 104 for 4 heads on each).  As in plain decode, a request is cut
// into splits of T tokens, and one CTA reduces one (request, value head,
// split); its warps take the split's 16-token chunks in turn, each through
// its own ring of stages filled by TMA.  The two heads of a value head lie
// side by side in a page, so one box brings K1 and K2 of a chunk and one
// both halves of V.
//
// One 16-row mma tile carries both maps: rows 0..7 are up to 8 heads' first
// map, rows 8..15 the same heads' second map.  Scores take one product with
// K1 (rows 0..7) and one with K2 (rows 8..15); the weights of both maps then
// meet V in the same product, so V is read from shared memory once for both.
// Each map has its own running maximum and sum, the difference is only
// taken when both are complete.
//
// Measured, both launches: 64 requests to 32K tokens, 4 value heads of 128, 368
// us against 358.5 for their bytes at the rate of a plain copy; one request
// of 250,001 on 4 of 64, 87 against 75; 16 of 1 to 4,097, 20.5 against 5.8,
// where the longest request's CTAs and the two launches' latency count. (Equal
// ranges over all requests, which each CTA finds from the lengths, were slower
// but for batches of equal lengths: 47 and 395 us for the ragged two, 52
// against 63 for 16 of 4,097 each.)
//
// Weights are split into bf16 terms, p = hi + lo (+ lo2 for fp32 outputs):
// 16 (24) bits of each weight.  The output is a difference of two averages
// that may nearly cancel, which would blow up the 2^-9 of a single term.
#include "phs_attn.cuh"
#include "phs_merge.cuh"
#include "phs_ops.h"

namespace phs {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// lambda of head i, by one warp
template <int D>
__device__ __forceinline__ float diff_lambda(const DiffArgs& a, int i, int lane) {
  const int off = a.lambda_per_head ? i * D : 0;
  float s1 = 0.f, s2 = 0.f;
#pragma unroll
  for (int d = lane; d < D; d += 32) {
    s1 = fmaf(__ldg(a.lambda_q1 + off + d), __ldg(a.lambda_k1 + off + d), s1);
    s2 = fmaf(__ldg(a.lambda_q2 + off + d), __ldg(a.lambda_k2 + off + d), s2);
  }
  return expf(warp_sum(s1)) - expf(warp_sum(s2)) + a.lambda_init;
}

// Difference, norm and store of head i by one warp: lane holds columns
// V lane .. V lane + V - 1 of both maps' sums o, and the sums l of weights.
template <int D>
__device__ __forceinline__ void finish_head(const DiffArgs& a, int b, int i, float lambda,
                                            const float (&o)[2][D / 16], const float (&l)[2],
                                            int lane) {
  constexpr int V = D / 16;
  // (a sum of NaN scores is NaN, and so is the row)
  const float i1 = l[0] == 0.f ? 0.f : 1.f / l[0], i2 = l[1] == 0.f ? 0.f : lambda / l[1];
  float x[V];
#pragma unroll
  for (int c = 0; c < V; ++c) x[c] = o[0][c] * i1 - o[1][c] * i2;
  if (a.norm_weight) {
    float sq = 0.f;
#pragma unroll
    for (int c = 0; c < V; ++c) sq = fmaf(x[c], x[c], sq);
    sq = warp_sum(sq);
    const float mean = sq / (2 * D) + a.norm_eps;
    const float f = mean == 0.f ? 0.f : (1.f - a.lambda_init) / sqrtf(mean);  // eps may be 0
#pragma unroll
    for (int c = 0; c < V; ++c) x[c] = x[c] * f * __ldg(a.norm_weight + V * lane + c);
  }
  const size_t at = (static_cast<size_t>(b) * a.H + i) * 2 * D + V * lane;
  if (a.out_f32) {
    float4* p = reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + at);
#pragma unroll
    for (int c = 0; c < V; c += 4) p[c / 4] = make_float4(x[c], x[c + 1], x[c + 2], x[c + 3]);
  } else {
    uint2* p = reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(a.out) + at);
#pragma unroll
    for (int c = 0; c < V; c += 4)
      p[c / 4] = make_uint2(pack_bf16(x[c], x[c + 1]), pack_bf16(x[c + 2], x[c + 3]));
  }
}

// Warps, stages and CTAs of an SM, by the time of a call in us (each at its
// best split length).  D = 128: 64 requests to 32K / one of 8K / 4 of 32K on
// one value head: 6 warps x 2 stages x 1 CTA 367 / 12.6 / 30.5, 3 x 2 x 2
// 371 / 14.8 / 34.2, 2 x 2 x 3 370 / 15.2 / 31.1.  D = 64: one of 250K / 32
// of 16K: 4 x 2 x 3 83.6 / 158.8, 4 x 3 x 2 85.8 / 161.3, 8 x 3 x 1
// 84.6 / 168.3.
template <int D>
struct DiffShape {
  static constexpr int NW = D == 128 ? 6 : 4;
  static constexpr int S = 2;
  static constexpr int kCtas = diff_ctas_per_sm(D);
};

template <int D>
struct DiffLayout {
  static constexpr int NW = DiffShape<D>::NW, S = DiffShape<D>::S, kCtas = DiffShape<D>::kCtas;
  static constexpr int kTile = 2 * kPage * D * 2;    // K1 and K2 (or V) of one chunk
  static constexpr int kStage = 2 * kTile;
  static constexpr int kMaxChunks = (kDiffMaxSplit / kPage + NW - 1) / NW;  // of a warp
  static constexpr int kIds = NW * S * kStage;
  static constexpr int kBar = kIds + NW * kMaxChunks * 4;
  static constexpr int kAlloc = kBar + NW * S * 8 + 1024;
  // the warps' results, over the stages once they are done
  static constexpr int kRow = 2 * D + 8;  // floats of a row: 32 bytes past a multiple of 128
  static constexpr int kO = NW * 16 * kRow;
  static_assert((kO + 2 * NW * 16) * 4 <= kIds, "results fit the stages");
};

// the running softmax of both maps and the output tile of one warp: rows g
// (map 1) and g + 8 (map 2) of its 16 x 2D tile
template <int D>
struct DiffState {
  float o[2 * D / 8][4];
  float m[2], l[2];
};

template <int D, int NT>
__device__ __forceinline__ void diff_chunk(DiffState<D>& st, const uint32_t (&qa)[D / 16][4],
                                           uint32_t sK, uint32_t sV, uint32_t valid,
                                           float scale_log2, int lane) {
  constexpr int kHalf = 2 * kPage * 128;  // bytes of 64 columns of a tile's 32 rows
  const int mi = lane >> 3, r = lane & 7, qd = lane & 3;
  float c[2][2][2];  // [map][8-token tile][score]
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) c[m][nt][0] = c[m][nt][1] = 0.f;
  // K fragments: matrix mi = tokens 8 (mi >> 1).., 16-byte unit 2 ks + (mi & 1)
  const uint32_t kb = sK + (r + 8 * (mi >> 1)) * 128 + ((((mi & 1) ^ r) & 7) << 4);
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks) {
    const uint32_t at = (kb ^ (((2 * ks) & 7) << 4)) + (ks >> 2) * kHalf;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      uint32_t b0, b1, b2, b3;
      ldsm_x4(at + m * kPage * 128, b0, b1, b2, b3);
      mma_bf16(c[m][0], qa[ks][m], 0u, qa[ks][2 + m], 0u, b0, b1);
      mma_bf16(c[m][1], qa[ks][m], 0u, qa[ks][2 + m], 0u, b2, b3);
    }
  }
  uint32_t pa[NT][4];
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    float x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 8 * (i >> 1) + 2 * qd + (i & 1);
      x[i] = ((valid >> t) & 1u) ? c[m][i >> 1][i & 1] : -INFINITY;
    }
    const float alpha = softmax_row_update(x, scale_log2, 0.f, 0.f, 1.f, st.m[m], st.l[m]);
    rescale_rows<2 * D, 4>(st.o, m, alpha);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t w = pack_bf16(x[2 * h], x[2 * h + 1]);
        pa[t][m + 2 * h] = w;
        x[2 * h] -= __uint_as_float(w << 16);
        x[2 * h + 1] -= __uint_as_float(w & 0xffff0000u);
      }
  }
  // V fragments (transposed): matrix mi = tokens 8 (mi & 1).., unit 2 np + (mi >> 1)
  const uint32_t vb = sV + (r + 8 * (mi & 1)) * 128 + ((((mi >> 1) ^ r) & 7) << 4);
#pragma unroll
  for (int hv = 0; hv < 2; ++hv)
#pragma unroll
    for (int np = 0; np < D / 16; ++np) {
      uint32_t v0, v1, v2, v3;
      ldsm_x4_t((vb ^ (((2 * np) & 7) << 4)) + (np >> 2) * kHalf + hv * kPage * 128, v0, v1, v2,
                v3);
      const int nt = hv * (D / 8) + 2 * np;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        mma_bf16(st.o[nt], pa[t][0], pa[t][1], pa[t][2], pa[t][3], v0, v1);
        mma_bf16(st.o[nt + 1], pa[t][0], pa[t][1], pa[t][2], pa[t][3], v2, v3);
      }
    }
}

template <int D, int NT>
__global__ void __launch_bounds__(DiffLayout<D>::NW * 32, DiffLayout<D>::kCtas)
    phs_diff_split_kernel(const __grid_constant__ CUtensorMap tk,
                          const __grid_constant__ CUtensorMap tv,
                          const __grid_constant__ DiffArgs a) {
  using L = DiffLayout<D>;
  constexpr int NW = L::NW, S = L::S, V = D / 16;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  pdl_launch_dependents();  // the merge may start; it waits for this grid
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, qd = lane & 3;
  // groups of more than 8 heads take two CTAs, 8 heads each
  const int gb = (a.G + 7) / 8, b = blockIdx.x, j = blockIdx.y / gb, g0 = 8 * (blockIdx.y % gb);
  const int s = blockIdx.z, live = min(8, a.G - g0), i0 = j * a.G + g0;
  int n = a.seq_lens[b];
  const bool appends = a.k_new != nullptr && n >= 1 && n <= a.n_clamp;
  if (n < 0 || n > a.n_clamp) {
    if (s == 0 && blockIdx.y == 0 && threadIdx.x == 0) set_status(a.status, PHS_ERANGE);
    n = max(0, min(n, a.n_clamp));
  }
  const int ns = (n + a.T - 1) / a.T;
  if (ns == 0) {
    const size_t row0 = (static_cast<size_t>(b) * a.H + i0) * 2 * D;
    if (s == 0)
      for (int e = threadIdx.x; e < live * 2 * D; e += NW * 32)
        store_out(a.out, row0 + e, 0.f, a.out_f32);
    return;
  }
  if (s >= ns) return;
  const int t0 = s * a.T, t1 = min(t0 + a.T, n);
  const int nch = (t1 - t0 + kPage - 1) / kPage;
  const int my_n = warp < nch ? (nch - warp + NW - 1) / NW : 0;

  int32_t* ids = reinterpret_cast<int32_t*>(smem + L::kIds) + warp * L::kMaxChunks;
  for (int c = lane; c < my_n; c += 32) {
    const int lp = t0 / kPage + warp + c * NW;
    int id = a.block_table[static_cast<size_t>(b) * a.max_pages + lp];
    if (id < 0 || id >= a.num_pages) {
      set_status(a.status, PHS_ERANGE);
      id = -1;
    }
    ids[c] = id;
  }
  const uint32_t bar0 = smem_u32(smem + L::kBar) + warp * S * 8;
  if (lane == 0) {
    for (int i = 0; i < S; ++i) mbar_init(bar0 + 8 * i, 1);
    fence_mbar_init();
  }
  __syncwarp();
  const uint32_t sbase = smem_u32(smem) + warp * S * L::kStage;
  const uint64_t pol = policy_evict_first();
  auto issue = [&](int c) {  // lane 0
    const uint32_t bar = bar0 + 8 * (c % S), dst = sbase + (c % S) * L::kStage;
    if (ids[c] < 0) {
      asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
      return;
    }
    mbar_arrive_expect_tx(bar, L::kStage);
    const int row = (ids[c] * a.Hv + j) * 2 * kPage;
    if constexpr (D == 128) {
      tma_load_3d(dst, &tk, 0, row, 0, bar, pol);
      tma_load_3d(dst + L::kTile, &tv, 0, row, 0, bar, pol);
    } else {
      tma_load_2d(dst, &tk, 0, row, bar, pol);
      tma_load_2d(dst + L::kTile, &tv, 0, row, bar, pol);
    }
  };
  // fused append: the warp whose chunk holds token n - 1 writes it into its
  // page before any of its copies is issued, and reads it back like the rest
  if (appends && n - 1 >= t0 && n - 1 < t1) {
    const int ci = (n - 1 - t0) / kPage;
    if (ci % NW == warp) {
      const int id = ids[ci / NW], r = (n - 1) % kPage;
      if (id >= 0) {
        if (a.page_refcount != nullptr && __ldg(a.page_refcount + id) != 1) {
          if (lane == 0) set_status(a.status, PHS_ESHARED);
        } else {
          const int op = lane >> 4, c = lane & 15;  // lanes 0-15 K, 16-31 V
          if (c < D / 8) {
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              const int h = 2 * j + m;
              const uint4 v = __ldg(reinterpret_cast<const uint4*>(
                  (op ? a.v_new : a.k_new) + (static_cast<size_t>(b) * 2 * a.Hv + h) * D + c * 8));
              *reinterpret_cast<uint4*>(
                  (op ? a.v : a.k) +
                  ((static_cast<size_t>(id) * 2 * a.Hv + h) * kPage + r) * D + c * 8) = v;
            }
            fence_proxy_async_global();
          }
        }
      }
      __syncwarp();
      if (lane == 0) fence_proxy_async_global();
    }
  }
  if (lane == 0)
    for (int c = 0; c < S && c < my_n; ++c) issue(c);

  // queries: rows g and g + 8 of the A tile are the two maps of head g
  uint32_t qa[D / 16][4];
  {
    const uint32_t* q = reinterpret_cast<const uint32_t*>(
        a.q + (static_cast<size_t>(b) * a.H + i0 + g) * 2 * D);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
      for (int f = 0; f < 4; ++f)  // f & 1: map, f >> 1: columns 8..15 of the step
        qa[ks][f] = g < live ? __ldg(q + (f & 1) * (D / 2) + 8 * ks + 4 * (f >> 1) + qd) : 0u;
  }
  DiffState<D> st;
#pragma unroll
  for (int i = 0; i < 2 * D / 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) st.o[i][e] = 0.f;
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    st.m[m] = -INFINITY;
    st.l[m] = 0.f;
  }
  int failed = -1;
  for (int c = 0; c < my_n; ++c) {
    if (!__all_sync(0xffffffffu, mbar_wait(bar0 + 8 * (c % S), (c / S) & 1))) {
      failed = c;
      break;
    }
    const uint32_t stage = sbase + (c % S) * L::kStage;
    if (ids[c] >= 0) {
      const int nv = t1 - (t0 + kPage * (warp + c * NW));
      const uint32_t valid = nv >= kPage ? 0xFFFFu : ((1u << nv) - 1u);
      if (valid != 0xFFFFu) {  // slots behind the last token: no NaN through 0 * V
        uint8_t* tile = smem + (stage + L::kTile - smem_u32(smem));
        for (int u = lane; u < L::kTile / 16; u += 32)
          if (!((valid >> ((u / 8) % kPage)) & 1u))
            *reinterpret_cast<uint4*>(tile + u * 16) = make_uint4(0, 0, 0, 0);
        __syncwarp();
      }
      diff_chunk<D, NT>(st, qa, stage, stage + L::kTile, valid, a.scale_log2, lane);
    }
    __syncwarp();
    if (lane == 0 && c + S < my_n) {
      fence_proxy_async_smem();
      issue(c + S);
    }
  }
  if (failed >= 0 && lane == 0) {  // record it and let the copies in flight land
    set_status(a.status, PHS_ETIMEOUT);
    for (int k = failed; k < my_n && k < failed + S; ++k)
      (void)mbar_wait(bar0 + 8 * (k % S), (k / S) & 1);
  }

  // ---- the warps' results meet in shared memory
  float lsum[2] = {warp_sum_quad(st.l[0]), warp_sum_quad(st.l[1])};
  __syncthreads();  // every warp is done with its stages
  float* sO = reinterpret_cast<float*>(smem);
  float* sM = sO + L::kO;
  float* sL = sM + NW * 16;
  if (g < live) {
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const int row = warp * 16 + 8 * m + g;
#pragma unroll
      for (int nt = 0; nt < 2 * D / 8; ++nt)
        *reinterpret_cast<float2*>(sO + row * L::kRow + 8 * nt + 2 * qd) =
            make_float2(st.o[nt][2 * m], st.o[nt][2 * m + 1]);
      if (qd == 0) {
        sM[row] = st.m[m];
        sL[row] = lsum[m];
      }
    }
  }
  __syncthreads();
  const size_t part = (static_cast<size_t>(b) * a.Hv + j) * a.max_splits + s;
  for (int h = warp; h < live; h += NW) {
    float o[2][V], l[2], M[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      M[m] = -INFINITY;
      l[m] = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) M[m] = fmaxf(M[m], sM[w * 16 + 8 * m + h]);
#pragma unroll
      for (int c = 0; c < V; ++c) o[m][c] = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const int row = w * 16 + 8 * m + h;
        const float f = sM[row] == -INFINITY ? 0.f : exp2f(sM[row] - M[m]);
        l[m] = fmaf(sL[row], f, l[m]);
#pragma unroll
        for (int c = 0; c < V; c += 4) {
          const float4 x = *reinterpret_cast<const float4*>(sO + row * L::kRow + V * lane + c);
          o[m][c] = fmaf(x.x, f, o[m][c]);
          o[m][c + 1] = fmaf(x.y, f, o[m][c + 1]);
          o[m][c + 2] = fmaf(x.z, f, o[m][c + 2]);
          o[m][c + 3] = fmaf(x.w, f, o[m][c + 3]);
        }
      }
    }
    if (ns == 1) {
      finish_head<D>(a, b, i0 + h, diff_lambda<D>(a, i0 + h, lane), o, l, lane);
    } else {
      const size_t row = part * a.G + g0 + h;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        float4* to = reinterpret_cast<float4*>(a.ws_o + (row * 2 + m) * 2 * D + V * lane);
#pragma unroll
        for (int c = 0; c < V; c += 4)
          to[c / 4] = make_float4(o[m][c], o[m][c + 1], o[m][c + 2], o[m][c + 3]);
        if (lane == 0)
          reinterpret_cast<float2*>(a.ws_ml)[row * 2 + m] = make_float2(M[m], l[m]);
      }
    }
  }
}

// Joins the splits of one (request, head): the CTA's warps take them in
// turn, with a running maximum of each map, and join in shared memory.
constexpr int kDiffMergeWarps = 4;

template <int D>
__global__ void __launch_bounds__(kDiffMergeWarps * 32)
    phs_diff_merge_kernel(const __grid_constant__ DiffArgs a) {
  constexpr int NW = kDiffMergeWarps, V = D / 16;
  __shared__ float sO[NW][2][2 * D], sM[NW][2], sL[NW][2];
  const int b = blockIdx.x, i = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = max(0, min(a.seq_lens[b], a.n_clamp)), ns = (n + a.T - 1) / a.T;
  if (ns <= 1) {  // (this grid must not end before the one in front of it)
    pdl_wait_prior_grid();
    return;
  }
  const float lambda = warp == 0 ? diff_lambda<D>(a, i, lane) : 0.f;
  const int j = i / a.G;
  const size_t row0 = (static_cast<size_t>(b) * a.Hv + j) * a.max_splits * a.G + i % a.G;
  pdl_wait_prior_grid();
  float o[2][V], M[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int c = 0; c < V; ++c) o[m][c] = 0.f;
  constexpr int U = 4;  // splits loaded together
  for (int s0 = warp; s0 < ns; s0 += NW * U) {
    float x[U][2][V];
    float2 ml[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int s = s0 + u * NW;
      const size_t row = row0 + static_cast<size_t>(min(s, ns - 1)) * a.G;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        ml[u][m] = s < ns ? reinterpret_cast<const float2*>(a.ws_ml)[row * 2 + m]
                          : make_float2(-INFINITY, 0.f);
        const float4* from =
            reinterpret_cast<const float4*>(a.ws_o + (row * 2 + m) * 2 * D + V * lane);
#pragma unroll
        for (int c = 0; c < V; c += 4) {
          const float4 y = from[c / 4];
          x[u][m][c] = y.x;
          x[u][m][c + 1] = y.y;
          x[u][m][c + 2] = y.z;
          x[u][m][c + 3] = y.w;
        }
      }
    }
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      float top = M[m];
#pragma unroll
      for (int u = 0; u < U; ++u) top = fmaxf(top, ml[u][m].x);
      if (top == -INFINITY) {  // nothing attended so far, or NaN scores alone
#pragma unroll
        for (int u = 0; u < U; ++u) l[m] += ml[u][m].y;  // zeros, or NaN
        continue;
      }
      const float keep = exp2f(M[m] - top);
      l[m] *= keep;
#pragma unroll
      for (int c = 0; c < V; ++c) o[m][c] *= keep;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float w = exp2f(ml[u][m].x - top);
        l[m] = fmaf(ml[u][m].y, w, l[m]);
#pragma unroll
        for (int c = 0; c < V; ++c) o[m][c] = fmaf(x[u][m][c], w, o[m][c]);
      }
      M[m] = top;
    }
  }
#pragma unroll
  for (int m = 0; m < 2; ++m) {
#pragma unroll
    for (int c = 0; c < V; ++c) sO[warp][m][V * lane + c] = o[m][c];
    if (lane == 0) {
      sM[warp][m] = M[m];
      sL[warp][m] = l[m];
    }
  }
  __syncthreads();
  if (warp != 0) return;
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    float top = sM[0][m];
#pragma unroll
    for (int w = 1; w < NW; ++w) top = fmaxf(top, sM[w][m]);
    l[m] = 0.f;
#pragma unroll
    for (int c = 0; c < V; ++c) o[m][c] = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float f = sM[w][m] == -INFINITY ? 0.f : exp2f(sM[w][m] - top);
      l[m] = fmaf(sL[w][m], f, l[m]);
#pragma unroll
      for (int c = 0; c < V; ++c) o[m][c] = fmaf(sO[w][m][V * lane + c], f, o[m][c]);
    }
  }
  finish_head<D>(a, b, i, lambda, o, l, lane);
}

template <int D, int NT>
static int launch_diff_t(const CUtensorMap& tk, const CUtensorMap& tv, const DiffArgs& a, int B,
                         cudaStream_t stream) {
  using L = DiffLayout<D>;
  auto kern = phs_diff_split_kernel<D, NT>;
  if (ensure_dynamic_smem(reinterpret_cast<const void*>(kern), L::kAlloc) != PHS_OK)
    return PHS_ECUDA;
  kern<<<dim3(B, a.Hv * ((a.G + 7) / 8), a.max_splits), L::NW * 32, L::kAlloc, stream>>>(tk, tv, a);
  if (cudaGetLastError() != cudaSuccess) return PHS_ECUDA;
  if (a.max_splits == 1) return PHS_OK;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(B, a.H);
  cfg.blockDim = dim3(kDiffMergeWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, phs_diff_merge_kernel<D>, a) == cudaSuccess ? PHS_OK : PHS_ECUDA;
}

int launch_diff_decode(int D, const CUtensorMap& tk, const CUtensorMap& tv, const DiffArgs& a,
                       int B, cudaStream_t stream) {
  if (D == 128)
    return a.out_f32 ? launch_diff_t<128, 3>(tk, tv, a, B, stream)
                     : launch_diff_t<128, 2>(tk, tv, a, B, stream);
  return a.out_f32 ? launch_diff_t<64, 3>(tk, tv, a, B, stream)
                   : launch_diff_t<64, 2>(tk, tv, a, B, stream);
}

}  // namespace phs
