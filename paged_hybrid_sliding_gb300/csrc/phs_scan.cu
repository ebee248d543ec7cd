// phs_scan.cu -- the selective scan of a state space layer for one new token
// per request or a few, over a pool of per-request states.
//
//   s   = softplus(dt + dt_bias)                       one step for each head and token
//   S_t = exp(s a) S_{t-1} + s x_t b_t^T               (P x N, fp32, one per head)
//   y_t = S_t c_t + skip x_t                           b, c shared by a group of heads
// with a <= 0 the head's rate.
#include "phs_common.cuh"
#include "phs_layers.h"
#include "phs_merge.cuh"
#include "phs_scan.cuh"

namespace phs {

namespace {

// Four bf16 as floats.
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u),
                     __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u));
}

// One CTA per (request, head): eight threads a row of the state, which is
// read, updated and written back in registers; a row's product with c meets
// in three shuffles.  The step reads and writes each state once and computes 2
// operations a byte, so it is bound by memory: 256 requests of 64 heads of 64 x
// 128 (1.08 GB) take 174 us, 161 for those bytes at the rate of a plain copy (191
// with the loads behind the check of the id; 232 with five CTAs an SM, whose
// registers do not hold a thread's loads; states of 128 x 128, 32 heads: 167 with
// two, 248 with four).
template <int P, int N>
__global__ void __launch_bounds__(256, P * N > 8192 ? 2 : 4)
    phs_scan_decode_kernel(const ScanArgs a) {
  constexpr int R = P / 32, V = N / 32;  // rows of a thread, float4s of a row
  const int b = blockIdx.x, h = blockIdx.y;
  const size_t orow = (static_cast<size_t>(b) * a.H + h) * P;
  const int r0 = threadIdx.x / 8, l = threadIdx.x % 8, g = h / (a.H / a.G);
  // the state is on its way while the request's id is checked against others
  const int64_t at = a.state_ids ? a.state_ids[b] : b;
  float4* S = reinterpret_cast<float4*>(a.state + (at * a.H + h) * P * N) + r0 * (N / 4) + l;
  float4 s[R][V];
  if (at >= 0 && at < a.num_states) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int v = 0; v < V; ++v) s[r][v] = S[r * 8 * N + 8 * v];
  }
  if (request_state(a, b) < 0) {
    if (threadIdx.x < P) store_out(a.out, orow + threadIdx.x, 0.f, a.out_f32);
    return;
  }
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

// The same for requests of up to kScanShort tokens, one after another while the
// state stays in registers (others are the chunks' launches'); the rows go out
// together at the end.  A chunk costs its whole time however few tokens it has,
// and a CTA of the chunks its start: 256 requests of 4 tokens, 64 heads of 64 x
// 128, take 253 us here (161 for their states' bytes), of 16 tokens 597, of 17,
// in chunks, 1,150.  Behind the chunks of longer requests, at whose end it fills
// the SMs: 16 of 1 to 517 tokens 67 us (70 with chunks alone; limits of 8, 16, 24
// and 32 tokens 67, 67, 66 and 72).  The limit of 16 is that call's; in a call of
// 256 requests chunks would first pay at about 35 tokens (29 us a token one by one).
template <int P, int N>
__global__ void __launch_bounds__(256, P * N > 8192 ? 2 : 3)
    phs_scan_short_kernel(const __grid_constant__ ScanArgs a) {
  constexpr int R = P / 32, V = N / 32;
  __shared__ float s_step[kScanShort], s_decay[kScanShort];
  __shared__ float s_y[kScanShort][P];
  const int b = blockIdx.x, h = blockIdx.y;
  const int64_t id = request_state(a, b);
  int t0, t1;
  const bool good = request_tokens(a, b, t0, t1);
  const int n = t1 - t0;
  if (!good || n > a.short_len) {
    pdl_wait_prior_grid();
    return;
  }
  if (id >= 0) {
    const int r0 = threadIdx.x / 8, l = threadIdx.x % 8, g = h / (a.H / a.G);
    float4* S = reinterpret_cast<float4*>(a.state + (id * a.H + h) * P * N) + r0 * (N / 4) + l;
    const bool resume = a.resume && a.resume[b] != 0;
    float4 s[R][V];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int v = 0; v < V; ++v)
        s[r][v] = resume ? S[r * 8 * N + 8 * v] : make_float4(0.f, 0.f, 0.f, 0.f);
    if (threadIdx.x < n) {
      const float step = scan_step(a, t0 + threadIdx.x, h);
      s_step[threadIdx.x] = step;
      s_decay[threadIdx.x] = decay_factor(step * a.rate[h]);
    }
    const float skip = a.skip ? a.skip[h] : 0.f;
    const __nv_bfloat16* bp = a.b + t0 * a.b_stride + g * N + 4 * l;
    const __nv_bfloat16* cp = a.c + t0 * a.c_stride + g * N + 4 * l;
    const __nv_bfloat16* xp = a.x + t0 * a.x_stride + h * P + r0;
    __syncthreads();
#pragma unroll 1
    for (int t = 0; t < n; ++t, bp += a.b_stride, cp += a.c_stride, xp += a.x_stride) {
      float4 bv[V], cv[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        bv[v] = load4(bp + 32 * v);
        cv[v] = load4(cp + 32 * v);
      }
      const float step = s_step[t], decay = s_decay[t];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float x = __bfloat162float(xp[32 * r]), sx = step * x;
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
        if (l == 0) s_y[t][r0 + 32 * r] = fmaf(skip, x, y);
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int v = 0; v < V; ++v) S[r * 8 * N + 8 * v] = s[r][v];
    __syncthreads();
  }
  uint32_t* out = reinterpret_cast<uint32_t*>(a.out) + (int64_t{t0} * a.H + h) * (P / 2);
  for (int e = threadIdx.x; e < n * (P / 2); e += 256) {
    const int t = e / (P / 2), p = e % (P / 2);
    out[static_cast<int64_t>(t) * a.H * (P / 2) + p] =
        id < 0 ? 0u : pack_bf16(s_y[t][2 * p], s_y[t][2 * p + 1]);
  }
  pdl_wait_prior_grid();  // (this grid's end must not come before that of the chunks' ones)
}

}  // namespace

int launch_scan_decode(int P, int N, const ScanArgs& a, cudaStream_t stream) {
  const dim3 grid(a.B, a.H);
  if (P == 128 && N == 128)
    phs_scan_decode_kernel<128, 128><<<grid, 256, 0, stream>>>(a);
  else if (P == 128)
    phs_scan_decode_kernel<128, 64><<<grid, 256, 0, stream>>>(a);
  else if (N == 128)
    phs_scan_decode_kernel<64, 128><<<grid, 256, 0, stream>>>(a);
  else
    phs_scan_decode_kernel<64, 64><<<grid, 256, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? PHS_OK : PHS_ECUDA;
}

int launch_scan_short(int P, int N, const ScanArgs& a, bool early, cudaStream_t stream) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = early;
  cfg.gridDim = dim3(a.B, a.H);
  cfg.blockDim = dim3(256);
  const cudaError_t err =
      P == 128 ? N == 128 ? cudaLaunchKernelEx(&cfg, phs_scan_short_kernel<128, 128>, a)
                          : cudaLaunchKernelEx(&cfg, phs_scan_short_kernel<128, 64>, a)
      : N == 128 ? cudaLaunchKernelEx(&cfg, phs_scan_short_kernel<64, 128>, a)
                 : cudaLaunchKernelEx(&cfg, phs_scan_short_kernel<64, 64>, a);
  if (err != cudaSuccess) return PHS_ECUDA;
  return cudaGetLastError() == cudaSuccess ? PHS_OK : PHS_ECUDA;
}

}  // namespace phs
