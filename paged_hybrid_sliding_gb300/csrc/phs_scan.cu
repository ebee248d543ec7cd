// phs_scan.cu -- the selective scan of a state space layer, over a pool of
// per-request states.
//
//   s   = softplus(dt + dt_bias)                       one step for each head and token
//   S_t = exp(s a) S_{t-1} + s x_t b_t^T               (P x N, fp32, one per head)
//   y_t = S_t c_t + skip x_t                           b, c shared by a group of heads
// with a <= 0 the head's rate.
#include "phs_common.cuh"
#include "phs_decay.cuh"
#include "phs_layers.h"
#include "phs_merge.cuh"

namespace phs {

namespace {

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

// Four bf16 as floats.
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u),
                     __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u));
}

// One CTA per (request, head): eight threads a row of the state, which is
// read, updated and written back in registers; a row's product with c meets
// in three shuffles.  The step reads and writes each state once and computes 2
// operations a byte, so it is bound by memory.
template <int P, int N>
__global__ void __launch_bounds__(256) phs_scan_decode_kernel(const ScanArgs a) {
  constexpr int R = P / 32, V = N / 32;  // rows of a thread, float4s of a row
  const int b = blockIdx.x, h = blockIdx.y;
  const int64_t id = scan_state(a, b);
  const size_t orow = (static_cast<size_t>(b) * a.H + h) * P;
  if (id < 0) {
    if (threadIdx.x < P) store_out(a.out, orow + threadIdx.x, 0.f, a.out_f32);
    return;
  }
  const int r0 = threadIdx.x / 8, l = threadIdx.x % 8, g = h / (a.H / a.G);
  float4* S = reinterpret_cast<float4*>(a.state + (id * a.H + h) * P * N) + r0 * (N / 4) + l;
  float4 s[R][V];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int v = 0; v < V; ++v) s[r][v] = S[r * 8 * N + 8 * v];
  const __nv_bfloat16* bp = a.b + b * a.b_stride + g * N + 4 * l;
  const __nv_bfloat16* cp = a.c + b * a.c_stride + g * N + 4 * l;
  float4 bv[V], cv[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    bv[v] = load4(bp + 32 * v);
    cv[v] = load4(cp + 32 * v);
  }
  const float step = scan_step(a, b, h), decay = decay_factor(step * a.rate[h]);
  const float skip = a.skip ? a.skip[h] : 0.f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int p = r0 + 32 * r;
    const float x = __bfloat162float(a.x[b * a.x_stride + h * P + p]), sx = step * x;
    float y = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float4& q = s[r][v];
      q.x = fmaf(sx, bv[v].x, decayed(q.x, decay));
      q.y = fmaf(sx, bv[v].y, decayed(q.y, decay));
      q.z = fmaf(sx, bv[v].z, decayed(q.z, decay));
      q.w = fmaf(sx, bv[v].w, decayed(q.w, decay));
      S[r * 8 * N + 8 * v] = q;
      y = fmaf(q.x, cv[v].x, fmaf(q.y, cv[v].y, fmaf(q.z, cv[v].z, fmaf(q.w, cv[v].w, y))));
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
    if (l == 0) store_out(a.out, orow + p, fmaf(skip, x, y), a.out_f32);
  }
}

// ------------------------------------------------------------- prompts --
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

// One CTA per (request, head), which walks the tokens with the state in
// registers, laid out as in the single step.
template <int P, int N>
__global__ void __launch_bounds__(256) phs_scan_prompt_kernel(const ScanArgs a) {
  constexpr int R = P / 32, V = N / 32;
  const int b = blockIdx.x, h = blockIdx.y, g = h / (a.H / a.G);
  const int64_t id = scan_state(a, b);
  int t0, t1;
  if (!scan_tokens(a, b, t0, t1)) return;
  __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.out) + h * P;
  const int64_t os = int64_t{a.H} * P;
  if (id < 0) {
    for (int t = t0; t < t1; ++t)
      if (threadIdx.x < P) out[t * os + threadIdx.x] = __float2bfloat16_rn(0.f);
    return;
  }
  const int r0 = threadIdx.x / 8, l = threadIdx.x % 8;
  float4* S = reinterpret_cast<float4*>(a.state + (id * a.H + h) * P * N) + r0 * (N / 4) + l;
  const bool resume = a.resume && a.resume[b] != 0;
  float4 s[R][V];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int v = 0; v < V; ++v)
      s[r][v] = resume ? S[r * 8 * N + 8 * v] : make_float4(0.f, 0.f, 0.f, 0.f);
  const float rate = a.rate[h], skip = a.skip ? a.skip[h] : 0.f;
  for (int t = t0; t < t1; ++t) {
    const float step = scan_step(a, t, h), decay = decay_factor(step * rate);
    const __nv_bfloat16* bp = a.b + t * a.b_stride + g * N + 4 * l;
    const __nv_bfloat16* cp = a.c + t * a.c_stride + g * N + 4 * l;
    float4 bv[V], cv[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      bv[v] = load4(bp + 32 * v);
      cv[v] = load4(cp + 32 * v);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int p = r0 + 32 * r;
      const float x = __bfloat162float(a.x[t * a.x_stride + h * P + p]), sx = step * x;
      float y = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float4& q = s[r][v];
        q.x = fmaf(sx, bv[v].x, decayed(q.x, decay));
        q.y = fmaf(sx, bv[v].y, decayed(q.y, decay));
        q.z = fmaf(sx, bv[v].z, decayed(q.z, decay));
        q.w = fmaf(sx, bv[v].w, decayed(q.w, decay));
        y = fmaf(q.x, cv[v].x, fmaf(q.y, cv[v].y, fmaf(q.z, cv[v].z, fmaf(q.w, cv[v].w, y))));
      }
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
      if (l == 0) out[t * os + p] = __float2bfloat16_rn(fmaf(skip, x, y));
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int v = 0; v < V; ++v) S[r * 8 * N + 8 * v] = s[r][v];
}

template <int P, int N>
int launch_scan_t(const ScanArgs& a, bool prompt, cudaStream_t stream) {
  const dim3 grid(a.B, a.H);
  if (prompt)
    phs_scan_prompt_kernel<P, N><<<grid, 256, 0, stream>>>(a);
  else
    phs_scan_decode_kernel<P, N><<<grid, 256, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? PHS_OK : PHS_ECUDA;
}

int launch_scan(int P, int N, const ScanArgs& a, bool prompt, cudaStream_t stream) {
  if (P == 128)
    return N == 128 ? launch_scan_t<128, 128>(a, prompt, stream)
                    : launch_scan_t<128, 64>(a, prompt, stream);
  return N == 128 ? launch_scan_t<64, 128>(a, prompt, stream)
                  : launch_scan_t<64, 64>(a, prompt, stream);
}

}  // namespace

int launch_scan_decode(int P, int N, const ScanArgs& a, cudaStream_t stream) {
  return launch_scan(P, N, a, false, stream);
}
int launch_scan_prompt(int P, int N, const ScanArgs& a, cudaStream_t stream) {
  return launch_scan(P, N, a, true, stream);
}

}  // namespace phs
