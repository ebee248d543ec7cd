// phs_conv.cu -- the short causal convolution of a selective state space
// layer, one filter of W = 2 to 4 taps for each channel:
//     y[t] = act(bias + sum_k weight[k] x[t - W + 1 + k])
// over packed prompts or one token per request, with the last W - 1 inputs of
// each channel kept between calls.
#include "phs_common.cuh"
#include "phs_layers.h"

namespace phs {

namespace {

constexpr int kConvTile = 32;  // tokens of a CTA

struct Vec {  // 8 channels
  float v[8];
};

__device__ __forceinline__ Vec unpack(const uint4& x) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&x);
  Vec r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.v[2 * i] = __uint_as_float(w[i] << 16);
    r.v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  return r;
}

// The channel's state, or -1 where the request has none: a negative id (an
// inactive request), one outside the pool, or one that an earlier request
// has.  All threads of the CTA call it.
__device__ __forceinline__ int64_t conv_state(const ConvArgs& a, int b) {
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

// A thread's filters.
template <int W>
struct Taps {
  float w[W][8], bias[8];
  __device__ __forceinline__ void load(const ConvArgs& a, int ch) {
    float f[8 * W];
#pragma unroll
    for (int i = 0; i < 2 * W; ++i)
      *reinterpret_cast<float4*>(f + 4 * i) =
          *reinterpret_cast<const float4*>(a.weight + static_cast<size_t>(ch) * W + 4 * i);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      bias[e] = a.bias ? a.bias[ch + e] : 0.f;
#pragma unroll
      for (int k = 0; k < W; ++k) w[k][e] = f[e * W + k];
    }
  }
  // h: the W - 1 inputs before x, oldest first
  __device__ __forceinline__ uint4 apply(const Vec (&h)[W - 1], const Vec& x, int silu) const {
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      y[e] = bias[e];
#pragma unroll
      for (int k = 0; k < W - 1; ++k) y[e] = fmaf(w[k][e], h[k].v[e], y[e]);
      y[e] = fmaf(w[W - 1][e], x.v[e], y[e]);
      // y / (1 + exp(-y)): exp overflows to infinity below -88, where y / inf
      // is the 0 that is wanted (and -inf / inf, the limit 0, is set)
      if (silu) y[e] = y[e] == -INFINITY ? 0.f : __fdividef(y[e], 1.f + ex2(-1.4426950408889634f * y[e]));
    }
    return make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]),
                      pack_bf16(y[6], y[7]));
  }
};

// One CTA per (some channels, request), a thread 8 channels.
template <int W>
__global__ void phs_conv_decode_kernel(const ConvArgs a) {
  const int b = blockIdx.y, vec = blockIdx.x * blockDim.x + threadIdx.x, vecs = a.channels / 8;
  const int64_t id = conv_state(a, b);
  if (vec >= vecs) return;
  uint4* out = reinterpret_cast<uint4*>(a.out) + static_cast<size_t>(b) * vecs + vec;
  if (id < 0) {
    *out = make_uint4(0, 0, 0, 0);
    return;
  }
  uint4* st = reinterpret_cast<uint4*>(a.state) + id * (W - 1) * vecs + vec;
  const uint4 x = *reinterpret_cast<const uint4*>(a.x + b * a.x_stride + 8 * vec);
  uint4 old[W - 1];
  Vec h[W - 1];
#pragma unroll
  for (int k = 0; k < W - 1; ++k) old[k] = st[static_cast<size_t>(k) * vecs];
  Taps<W> taps;
  taps.load(a, 8 * vec);
#pragma unroll
  for (int k = 0; k < W - 1; ++k) h[k] = unpack(old[k]);
  *out = taps.apply(h, unpack(x), a.silu);
#pragma unroll
  for (int k = 0; k < W - 1; ++k) st[static_cast<size_t>(k) * vecs] = k + 1 < W - 1 ? old[k + 1] : x;
}

// One CTA per (tile of 32 packed rows, some channels), a thread 8 channels of
// the tile's rows in order, the W - 1 inputs before a row in registers.  A
// request's first W - 1 rows, whose inputs reach into the pool, and the pool's
// update belong to the tile that its first row is in, whatever tiles those
// rows are in: its old inputs are read before the thread that owns them writes
// the new ones.
template <int W>
__global__ void phs_conv_prompt_kernel(const ConvArgs a) {
  __shared__ int s_b0, s_b1;  // requests that begin in the tile or reach into it
  const int vec = blockIdx.x * blockDim.x + threadIdx.x, vecs = a.channels / 8;
  const bool mine = vec < vecs;
  const int r0 = blockIdx.y * kConvTile, r1 = min(r0 + kConvTile, a.tokens);
  const bool last_tile = r1 == a.tokens;
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
  Taps<W> taps;
  if (mine) taps.load(a, 8 * vec);
  const uint4* x = reinterpret_cast<const uint4*>(a.x + 8 * vec);
  const int64_t xs = a.x_stride / 8;
  uint4* out = reinterpret_cast<uint4*>(a.out) + vec;
  for (int b = s_b0; b < s_b1; ++b) {
    const int lo = a.cu_seqlens[b], hi = a.cu_seqlens[b + 1];
    const int64_t id = conv_state(a, b);
    if (!mine) continue;
    const bool begins = lo >= r0;
    // this tile's rows of the request
    const int t0 = begins ? lo : max(r0, lo + W - 1);
    const int t1 = begins ? min(hi, max(r1, lo + W - 1)) : min(hi, r1);
    if (id < 0) {
      for (int t = t0; t < t1; ++t) out[static_cast<size_t>(t) * vecs] = make_uint4(0, 0, 0, 0);
      continue;
    }
    const bool resume = a.resume && a.resume[b] != 0;
    uint4* st = reinterpret_cast<uint4*>(a.state) + id * (W - 1) * vecs + vec;
    uint4 old[W - 1];
    Vec h[W - 1];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
      old[k] = make_uint4(0, 0, 0, 0);
      if (!begins) {
        if (t0 < t1) old[k] = x[(t0 - (W - 1) + k) * xs];
      } else if (resume) {
        old[k] = st[static_cast<size_t>(k) * vecs];
      }
      h[k] = unpack(old[k]);
    }
    int t = t0;
    for (; t + 4 <= t1; t += 4) {  // four rows' loads at once
      uint4 y[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = x[(t + j) * xs];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const Vec now = unpack(y[j]);
        out[static_cast<size_t>(t + j) * vecs] = taps.apply(h, now, a.silu);
#pragma unroll
        for (int k = 0; k < W - 1; ++k) h[k] = k + 1 < W - 1 ? h[k + 1] : now;
      }
    }
    for (; t < t1; ++t) {
      const Vec now = unpack(x[t * xs]);
      out[static_cast<size_t>(t) * vecs] = taps.apply(h, now, a.silu);
#pragma unroll
      for (int k = 0; k < W - 1; ++k) h[k] = k + 1 < W - 1 ? h[k + 1] : now;
    }
    if (begins) {  // the last W - 1 inputs
      const int n = hi - lo;
#pragma unroll
      for (int k = 0; k < W - 1; ++k) {
        const int i = n + k;  // of the old inputs and the new ones behind them
        uint4 y = make_uint4(0, 0, 0, 0);
        if (i >= W - 1)
          y = x[(lo + i - (W - 1)) * xs];
        else
#pragma unroll
          for (int m = 0; m < W - 1; ++m)
            if (m == i) y = old[m];
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
int launch_conv_t(const ConvArgs& a, bool prompt, cudaStream_t stream) {
  const int vecs = a.channels / 8, threads = 32 * conv_warps(vecs);
  const int blocks = (vecs + threads - 1) / threads;
  if (prompt) {
    const int tiles = a.tokens > 0 ? (a.tokens + kConvTile - 1) / kConvTile : 1;
    phs_conv_prompt_kernel<W><<<dim3(blocks, tiles), threads, 0, stream>>>(a);
  } else {
    phs_conv_decode_kernel<W><<<dim3(blocks, a.B), threads, 0, stream>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? PHS_OK : PHS_ECUDA;
}

int launch_conv(int width, const ConvArgs& a, bool prompt, cudaStream_t stream) {
  return width == 4   ? launch_conv_t<4>(a, prompt, stream)
         : width == 3 ? launch_conv_t<3>(a, prompt, stream)
                      : launch_conv_t<2>(a, prompt, stream);
}

}  // namespace

int launch_conv_decode(int width, const ConvArgs& a, cudaStream_t stream) {
  return launch_conv(width, a, false, stream);
}
int launch_conv_prompt(int width, const ConvArgs& a, cudaStream_t stream) {
  return launch_conv(width, a, true, stream);
}

}  // namespace phs
