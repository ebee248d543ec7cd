// phs_linear.cu -- linear attention with a decay for each head, over a pool
// of per-request states.
//
//   S_t = exp(g_h) S_{t-1} + k_t v_t^T        (D x D, fp32, one per KV head)
//   o_t = scale q_t^T S_t                     (every query head of the group)
// with g_h <= 0 the head's log decay.
#include "phs_common.cuh"
#include "phs_merge.cuh"
#include "phs_ops.h"

namespace phs {

// exp(g) s as s + (exp(g) - 1) s: the rounding of exp(g) itself, off by up to
// 2^-25, would come back in every step and grow with the memory of the head
// (a rate of 2e-4 holds 5,000 tokens: 1.5e-4 of the state).
__device__ __forceinline__ float decayed(float s, float expm1_g) { return fmaf(s, expm1_g, s); }

// The state of request b, or -1 where it has none: a negative id (an
// inactive request), one outside the pool, or one that an earlier request
// of the call has (two requests must not update one state).  All threads of
// the CTA call it.
__device__ __forceinline__ int64_t request_state(const LinearArgs& a, int b) {
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

// The token range of request b of a prompt call; false where it is bad: outside
// the tokens, longer than stated, or beginning before the end of an earlier
// one (two requests must not write one row).  All threads of the CTA call it.
__device__ __forceinline__ bool request_tokens(const LinearArgs& a, int b, int& t0, int& t1) {
  t0 = a.cu_seqlens[b];
  t1 = a.cu_seqlens[b + 1];
  int bad = t0 < 0 || t1 < t0 || t1 > a.total_tokens || t1 - t0 > a.max_seq;
  for (int j = threadIdx.x; j < b; j += blockDim.x) bad |= a.cu_seqlens[j] > t0;
  bad = __syncthreads_or(bad);
  if (bad && threadIdx.x == 0) set_status(a.status, PHS_ERANGE);
  return !bad;
}

// One CTA per (request, KV head).  A row of the state (one k index) is D/4
// threads of one float4 each.
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
  const float decay = expm1f(a.log_decay[h]);
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

// The recurrence token by token: one CTA per (16 columns of v, KV head,
// request).  Eight threads share a column, each with D/8 rows of the state
// in registers.
template <int D>
__global__ void __launch_bounds__(128) phs_linear_prompt_kernel(const LinearArgs a) {
  constexpr int R = D / 8;
  const int b = blockIdx.x, h = blockIdx.y, c0 = blockIdx.z * 16;
  const int col = threadIdx.x / 8, part = threadIdx.x % 8;
  const int64_t id = request_state(a, b);
  int t0, t1;
  if (!request_tokens(a, b, t0, t1)) return;
  if (id < 0) {
    for (int t = t0; t < t1; ++t)
      for (int g = part; g < a.G; g += 8)
        store_out(a.out, (static_cast<size_t>(t) * a.Hq + h * a.G + g) * D + c0 + col, 0.f,
                  a.out_f32);
    return;
  }
  float* S = a.state + (id * a.Hkv + h) * D * D;
  const float decay = expm1f(a.log_decay[h]);
  const bool resume = a.resume && a.resume[b] != 0;
  float s[R];
#pragma unroll
  for (int r = 0; r < R; ++r) s[r] = resume ? S[(part + 8 * r) * D + c0 + col] : 0.f;
  for (int t = t0; t < t1; ++t) {
    const __nv_bfloat16* k = a.k + (static_cast<size_t>(t) * a.Hkv + h) * D;
    const float v = __bfloat162float(a.v[(static_cast<size_t>(t) * a.Hkv + h) * D + c0 + col]);
#pragma unroll
    for (int r = 0; r < R; ++r)
      s[r] = fmaf(__bfloat162float(k[part + 8 * r]), v, decayed(s[r], decay));
    for (int g = 0; g < a.G; ++g) {
      const size_t row = (static_cast<size_t>(t) * a.Hq + h * a.G + g) * D;
      float x = 0.f;
#pragma unroll
      for (int r = 0; r < R; ++r) x = fmaf(__bfloat162float(a.q[row + part + 8 * r]), s[r], x);
      x += __shfl_xor_sync(0xffffffffu, x, 1);
      x += __shfl_xor_sync(0xffffffffu, x, 2);
      x += __shfl_xor_sync(0xffffffffu, x, 4);
      if (part == 0) store_out(a.out, row + c0 + col, x * a.scale, a.out_f32);
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) S[(part + 8 * r) * D + c0 + col] = s[r];
}

int launch_linear_prompt(int D, const LinearArgs& a, cudaStream_t stream) {
  const dim3 grid(a.B, a.Hkv, D / 16);
  if (D == 128)
    phs_linear_prompt_kernel<128><<<grid, 128, 0, stream>>>(a);
  else
    phs_linear_prompt_kernel<64><<<grid, 128, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? PHS_OK : PHS_ECUDA;
}

}  // namespace phs
