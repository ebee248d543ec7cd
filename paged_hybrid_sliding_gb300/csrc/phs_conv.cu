// phs_conv.cu -- the short causal convolution of a selective state space
// layer, one filter of W = 2 to 4 taps for each channel:
//     y[t] = act(bias + sum_k weight[k] x[t - W + 1 + k])
// over packed prompts or one token per request, with the last W - 1 inputs of
// each channel kept between calls.
#include "phs_layers.h"
#include "phs_prompt.cuh"
#include "phs_request.cuh"

namespace phs {

namespace {

// A thread takes four channels: with eight its filters and inputs hold the
// registers that loads in flight need (32,751 rows of 6,144 channels: 149 us,
// 156 with eight).
constexpr int kChan = 4;
constexpr int kRows = 8;  // whose loads are in flight while as many are summed up

struct Vec {  // in pairs
  uint64_t v[kChan / 2];
};

__device__ __forceinline__ Vec unpack(const uint2& x) {
  Vec r;
  r.v[0] = f2(x.x << 16, x.x & 0xFFFF0000u);
  r.v[1] = f2(x.y << 16, x.y & 0xFFFF0000u);
  return r;
}

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A thread's filters.
template <int W>
struct Taps {
  uint64_t w[W][kChan / 2], bias[kChan / 2];
  __device__ __forceinline__ void load(const ConvArgs& a, int ch) {
    float f[kChan * W];
#pragma unroll
    for (int i = 0; i < W; ++i)
      *reinterpret_cast<float4*>(f + 4 * i) =
          *reinterpret_cast<const float4*>(a.weight + static_cast<size_t>(ch) * W + 4 * i);
    float4 b = make_float4(0.f, 0.f, 0.f, 0.f);
    if (a.bias) b = *reinterpret_cast<const float4*>(a.bias + ch);
    bias[0] = f2(b.x, b.y);
    bias[1] = f2(b.z, b.w);
#pragma unroll
    for (int e = 0; e < kChan / 2; ++e)
#pragma unroll
      for (int k = 0; k < W; ++k) w[k][e] = f2(f[2 * e * W + k], f[(2 * e + 1) * W + k]);
  }
  // h: the W - 1 inputs before x, oldest first
  __device__ __forceinline__ uint2 apply(const Vec (&h)[W - 1], const Vec& x, int silu) const {
    uint32_t o[kChan / 2];
#pragma unroll
    for (int e = 0; e < kChan / 2; ++e) {
      uint64_t y = bias[e];
#pragma unroll
      for (int k = 0; k < W - 1; ++k) y = f2_fma(w[k][e], h[k].v[e], y);
      y = f2_fma(w[W - 1][e], x.v[e], y);
      if (silu) {
        // y / (1 + exp(-y)): below -87.3 the reciprocal is flushed to zero (the
        // quotient is above -1.1e-36 there), of -infinity too, whose limit is 0: that
        // factor is cut at the lowest number, a NaN comes in by the other one
        const float2 z = f2_get(f2_mul(y, f2(-1.4426950408889634f, -1.4426950408889634f)));
        const float2 d = f2_get(f2_add(f2(ex2(z.x), ex2(z.y)), f2(1.f, 1.f))), v = f2_get(y);
        y = f2_mul(f2(fmaxf(v.x, -3.402823466e38f), fmaxf(v.y, -3.402823466e38f)),
                   f2(rcp(d.x), rcp(d.y)));
      }
      o[e] = pack_term(y);
    }
    return make_uint2(o[0], o[1]);
  }
};

// One CTA per (some channels, request), a thread four channels.
template <int W>
__global__ void phs_conv_decode_kernel(const ConvArgs a) {
  const int b = blockIdx.y, vec = blockIdx.x * blockDim.x + threadIdx.x, vecs = a.channels / kChan;
  const int64_t id = request_state(a, b);
  if (vec >= vecs) return;
  uint2* out = reinterpret_cast<uint2*>(a.out) + static_cast<size_t>(b) * vecs + vec;
  if (id < 0) {
    *out = make_uint2(0, 0);
    return;
  }
  uint2* st = reinterpret_cast<uint2*>(a.state) + id * (W - 1) * vecs + vec;
  const uint2 x = *reinterpret_cast<const uint2*>(a.x + b * a.x_stride + kChan * vec);
  uint2 old[W - 1];
  Vec h[W - 1];
#pragma unroll
  for (int k = 0; k < W - 1; ++k) old[k] = st[static_cast<size_t>(k) * vecs];
  Taps<W> taps;
  taps.load(a, kChan * vec);
#pragma unroll
  for (int k = 0; k < W - 1; ++k) h[k] = unpack(old[k]);
  *out = taps.apply(h, unpack(x), a.silu);
#pragma unroll
  for (int k = 0; k < W - 1; ++k)
    st[static_cast<size_t>(k) * vecs] = k + 1 < W - 1 ? old[k + 1] : x;
}

// One CTA per (tile of packed rows, some channels), a thread four channels of the
// tile's rows in order, the W - 1 inputs before a row in registers.  A
// request's first W - 1 rows, whose inputs reach into the pool, and the pool's
// update belong to the tile that its first row is in, whatever tiles those
// rows are in: its old inputs are read before the thread that owns them writes
// the new ones.
//
// Each row is read and written once, with two operations of the special-function
// unit a value: 32,751 rows of 6,144 channels take 149 us, 120 for their bytes, 80
// of that unit's time.  (216 with sums one value at a time and no rows ahead; 161
// with four rows ahead, 156 and 164 with tiles of 64 and 256 rows.)
template <int W>
__global__ void __launch_bounds__(256, 2) phs_conv_prompt_kernel(const ConvArgs a, int tile) {
  __shared__ int s_b0, s_b1;  // requests that begin in the tile or reach into it
  const int vec = blockIdx.x * blockDim.x + threadIdx.x, vecs = a.channels / kChan;
  const bool mine = vec < vecs;
  const int r0 = blockIdx.y * tile, r1 = min(r0 + tile, a.tokens);
  const bool last_tile = r1 == a.tokens;
  Taps<W> taps;
  if (mine) taps.load(a, kChan * vec);
  if (threadIdx.x == 0) {
    s_b0 = a.B;
    s_b1 = 0;
  }
  __syncthreads();
  int bad = 0;
  for (int j = threadIdx.x; j < a.B; j += blockDim.x) {
    const int lo = a.cu_seqlens[j], hi = a.cu_seqlens[j + 1];
    bad |= lo < 0 || hi < lo || hi > a.tokens;
    // (an empty request behind the last row begins in the last tile)
    const bool begins = lo >= r0 && (lo < r1 || last_tile);
    if (begins || (lo < r0 && hi > r0)) {
      atomicMin(&s_b0, j);
      atomicMax(&s_b1, j + 1);
    }
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) set_status(a.status, PHS_ERANGE);
    return;
  }
  const uint2* x = reinterpret_cast<const uint2*>(a.x + kChan * vec);
  const int64_t xs = a.x_stride / kChan;
  uint2* out = reinterpret_cast<uint2*>(a.out) + vec;
  for (int b = s_b0; b < s_b1; ++b) {
    const int lo = a.cu_seqlens[b], hi = a.cu_seqlens[b + 1];
    const int64_t id = request_state(a, b);
    if (!mine) continue;
    const bool begins = lo >= r0;
    // this tile's rows of the request
    const int t0 = begins ? lo : max(r0, lo + W - 1);
    const int t1 = begins ? min(hi, max(r1, lo + W - 1)) : min(hi, r1);
    if (id < 0) {
      for (int t = t0; t < t1; ++t) out[static_cast<size_t>(t) * vecs] = make_uint2(0, 0);
      continue;
    }
    const bool resume = a.resume && a.resume[b] != 0;
    uint2* st = reinterpret_cast<uint2*>(a.state) + id * (W - 1) * vecs + vec;
    uint2 old[W - 1], ahead[kRows];
    auto read = [&](int t) {
#pragma unroll
      for (int j = 0; j < kRows; ++j)
        if (t + j < t1) ahead[j] = x[(t + j) * xs];
    };
    read(t0);
    Vec h[W - 1];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
      old[k] = make_uint2(0, 0);
      if (!begins) {
        if (t0 < t1) old[k] = x[(t0 - (W - 1) + k) * xs];
      } else if (resume) {
        old[k] = st[static_cast<size_t>(k) * vecs];
      }
      h[k] = unpack(old[k]);
    }
    for (int t = t0; t < t1; t += kRows) {
      uint2 now[kRows];
#pragma unroll
      for (int j = 0; j < kRows; ++j) now[j] = ahead[j];
      read(t + kRows);
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        if (t + j >= t1) break;
        const Vec y = unpack(now[j]);
        out[static_cast<size_t>(t + j) * vecs] = taps.apply(h, y, a.silu);
#pragma unroll
        for (int k = 0; k < W - 1; ++k) h[k] = k + 1 < W - 1 ? h[k + 1] : y;
      }
    }
    if (begins) {  // the last W - 1 inputs
      const int n = hi - lo;
#pragma unroll
      for (int k = 0; k < W - 1; ++k) {
        const int i = n + k;  // of the old inputs and the new ones behind them
        uint2 y = make_uint2(0, 0);
        if (i >= W - 1)
          y = x[(lo + i - (W - 1)) * xs];
        else if (resume)
          y = st[static_cast<size_t>(i) * vecs];  // (above k: not yet overwritten)
        st[static_cast<size_t>(k) * vecs] = y;
      }
    }
  }
}

// Warps of a CTA for `vecs` threads: the number from 4 to 8 that leaves the
// fewest threads idle.
int conv_warps(int vecs) {
  const int warps = (vecs + 31) / 32;
  int best = warps < 4 ? warps : 4, waste = INT32_MAX;
  for (int w = best; w <= 8 && w <= warps; ++w) {
    const int idle = (warps + w - 1) / w * w - warps;
    if (idle < waste) {
      waste = idle;
      best = w;
    }
  }
  return best;
}

template <int W>
int launch_conv_t(const ConvArgs& a, bool prompt, int num_sms, cudaStream_t stream) {
  const int vecs = a.channels / kChan, threads = 32 * conv_warps(vecs);
  const int blocks = (vecs + threads - 1) / threads;
  if (prompt) {
    // Longer tiles spread a CTA's start over more rows, as long as there are
    // eight CTAs an SM.
    int tile = 128;
    while (tile > 16 && int64_t{a.tokens} * blocks < int64_t{8} * num_sms * tile) tile /= 2;
    while (a.tokens > 65535 * int64_t{tile}) tile *= 2;  // grid y
    const int tiles = a.tokens > 0 ? (a.tokens + tile - 1) / tile : 1;
    phs_conv_prompt_kernel<W><<<dim3(blocks, tiles), threads, 0, stream>>>(a, tile);
  } else {
    phs_conv_decode_kernel<W><<<dim3(blocks, a.B), threads, 0, stream>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? PHS_OK : PHS_ECUDA;
}

int launch_conv(int width, const ConvArgs& a, bool prompt, int num_sms, cudaStream_t stream) {
  return width == 4   ? launch_conv_t<4>(a, prompt, num_sms, stream)
         : width == 3 ? launch_conv_t<3>(a, prompt, num_sms, stream)
                      : launch_conv_t<2>(a, prompt, num_sms, stream);
}

}  // namespace

int launch_conv_decode(int width, const ConvArgs& a, cudaStream_t stream) {
  return launch_conv(width, a, false, 0, stream);
}
int launch_conv_prompt(int width, const ConvArgs& a, int num_sms, cudaStream_t stream) {
  return launch_conv(width, a, true, num_sms, stream);
}

}  // namespace phs
