// phs_request.cuh -- what the recurrent layers' kernels (linear attention, the
// causal convolution, the selective scan) ask of a call's requests.
#pragma once

#include "phs_common.cuh"

namespace phs {

// The state of request b, or -1 where it has none: a negative id (an
// inactive request), one outside the pool, or one that an earlier request
// of the call has (two requests must not update one state).  All threads of
// the CTA call it.
template <class Args>
__device__ __forceinline__ int64_t request_state(const Args& a, int b) {
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

// The token range of request b; false where it is bad: outside the tokens,
// longer than stated, or beginning before the end of an earlier one (two
// requests must not write one row).  All threads of the CTA call it.
template <class Args>
__device__ __forceinline__ bool request_tokens(const Args& a, int b, int& t0, int& t1) {
  t0 = a.cu_seqlens[b];
  t1 = a.cu_seqlens[b + 1];
  int bad = t0 < 0 || t1 < t0 || t1 > a.total_tokens || t1 - t0 > a.max_seq;
  for (int j = threadIdx.x; j < b; j += blockDim.x) bad |= a.cu_seqlens[j] > t0;
  bad = __syncthreads_or(bad);
  if (bad && threadIdx.x == 0) set_status(a.status, PHS_ERANGE);
  return !bad;
}

// First chunk of part p of a request's `chunks`; a segment is nsub parts, and
// part nseg * nsub is the end.
template <class Args>
__device__ __forceinline__ int part_chunk(const Args& a, int chunks, int p) {
  return static_cast<int>(static_cast<int64_t>(chunks) * p / (a.nseg * a.nsub));
}

}  // namespace phs
