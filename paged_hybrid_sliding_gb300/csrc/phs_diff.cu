// phs_diff.cu -- differential attention of one new token per request over
// the paged pool.
//
//   out_i = (softmax(s q_{2i} K1) - lambda softmax(s q_{2i+1} K2)) V
//   lambda = exp(lambda_q1 . lambda_k1) - exp(lambda_q2 . lambda_k2) + lambda_init
// and, with a norm weight g,
//   out_i <- (1 - lambda_init) g out_i / sqrt(mean(out_i^2) + eps).
// Value head j of head i (j = i / (H / Hv)) has the two keys in pool heads
// 2j and 2j + 1 of K, and its 2D value columns in the same two heads of V.
#include "phs_common.cuh"
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
  for (int d = lane; d < D; d += 32) {
    s1 = fmaf(a.lambda_q1[off + d], a.lambda_k1[off + d], s1);
    s2 = fmaf(a.lambda_q2[off + d], a.lambda_k2[off + d], s2);
  }
  return expf(warp_sum(s1)) - expf(warp_sum(s2)) + a.lambda_init;
}

// One CTA per (request, head): its 8 warps take the tokens in turn, each with
// a running softmax of both maps; the warps' states join in shared memory.
template <int D>
__global__ void __launch_bounds__(256) phs_diff_decode_kernel(const DiffArgs a) {
  constexpr int NW = 8, V = D / 32, O = 2 * D / 32;
  __shared__ float sO[2][NW][2 * D];
  __shared__ float sM[2][NW], sL[2][NW], sSq[NW];
  const int b = blockIdx.x, i = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int j = i / a.G;
  int n = a.seq_lens[b];
  if (n < 0 || n > a.n_clamp) {
    if (threadIdx.x == 0) set_status(a.status, PHS_ERANGE);
    n = max(0, min(n, a.n_clamp));
  }
  float q[2][V], o[2][O], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int e = 0; e < 2; ++e) {
#pragma unroll
    for (int c = 0; c < V; ++c)
      q[e][c] = __bfloat162float(
          a.q[((static_cast<size_t>(b) * a.H + i) * 2 + e) * D + lane + 32 * c]);
#pragma unroll
    for (int c = 0; c < O; ++c) o[e][c] = 0.f;
  }
  for (int t = warp; t < n; t += NW) {
    const int page = a.block_table[static_cast<size_t>(b) * a.max_pages + t / kPage];
    if (page < 0 || page >= a.num_pages) {
      set_status(a.status, PHS_ERANGE);
      continue;
    }
    float v[O];
    size_t row[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      row[e] = ((static_cast<size_t>(page) * 2 * a.Hv + 2 * j + e) * kPage + t % kPage) * D;
#pragma unroll
      for (int c = 0; c < V; ++c) v[e * V + c] = __bfloat162float(a.v[row[e] + lane + 32 * c]);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float s = 0.f;
#pragma unroll
      for (int c = 0; c < V; ++c)
        s = fmaf(q[e][c], __bfloat162float(a.k[row[e] + lane + 32 * c]), s);
      s = warp_sum(s) * a.scale_log2;
      const float mn = fmaxf(m[e], s);
      const float keep = exp2f(m[e] - mn), p = exp2f(s - mn);
      l[e] = l[e] * keep + p;
#pragma unroll
      for (int c = 0; c < O; ++c) o[e][c] = fmaf(p, v[c], o[e][c] * keep);
      m[e] = mn;
    }
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
#pragma unroll
    for (int c = 0; c < O; ++c) sO[e][warp][lane + 32 * c] = o[e][c];
    if (lane == 0) {
      sM[e][warp] = m[e];
      sL[e][warp] = l[e];
    }
  }
  __syncthreads();
  const float lambda = diff_lambda<D>(a, i, lane);
  const int c = threadIdx.x;  // output column
  float r = 0.f;
  if (c < 2 * D) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float M = -INFINITY, L = 0.f, x = 0.f;
      for (int w = 0; w < NW; ++w) M = fmaxf(M, sM[e][w]);
      for (int w = 0; w < NW; ++w) {
        const float f = sM[e][w] == -INFINITY ? 0.f : exp2f(sM[e][w] - M);
        L = fmaf(sL[e][w], f, L);
        x = fmaf(sO[e][w][c], f, x);
      }
      x = L > 0.f ? x / L : 0.f;
      r = e ? r - lambda * x : x;
    }
  }
  if (a.norm_weight) {
    const float sq = warp_sum(r * r);
    if (lane == 0) sSq[warp] = sq;
    __syncthreads();
    float sum = 0.f;
    for (int w = 0; w < NW; ++w) sum += sSq[w];
    if (c < 2 * D)
      r *= a.norm_weight[c] * (1.f - a.lambda_init) / sqrtf(sum / (2 * D) + a.norm_eps);
  }
  if (c < 2 * D) store_out(a.out, (static_cast<size_t>(b) * a.H + i) * 2 * D + c, r, a.out_f32);
}

int launch_diff_decode(int D, const DiffArgs& a, int B, cudaStream_t stream) {
  if (D == 128)
    phs_diff_decode_kernel<128><<<dim3(B, a.H), 256, 0, stream>>>(a);
  else
    phs_diff_decode_kernel<64><<<dim3(B, a.H), 256, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? PHS_OK : PHS_ECUDA;
}

}  // namespace phs
