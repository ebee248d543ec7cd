// phs_pages.cu -- device-side page operations of a paged cache: freeing and
// forking requests and compacting the pool, with the block tables, lengths
// and reference counts that the decode kernels read kept on the device (no
// host round trip, recordable into a graph).
//
// Everything here is integer bookkeeping and byte copies.  Results do not
// depend on the order of atomics: counts are sums, and every choice of a
// page goes by rank in page order (the lowest free pages to the forks in
// their order; the highest live page to the lowest hole).
#include "phs_common.cuh"
#include "phs_ops.h"

namespace phs {

// A request's pages inside its table row; lengths outside the table are an
// error and hold no pages here.
__device__ __forceinline__ int held_pages(int n, int max_pages, int32_t* status) {
  if (n < 0 || n > max_pages * kPage) {
    set_status(status, PHS_ERANGE);
    return 0;
  }
  return (n + kPage - 1) / kPage;
}

// ------------------------------------------------------------------ free --
// One CTA per listed row: one reference less on each of its pages, then the
// row's length is zero.
__global__ void __launch_bounds__(256) phs_pages_free_kernel(const PageFreeArgs a) {
  const int i = blockIdx.x, r = a.rows[i];
  int bad = r < 0 || r >= a.num_rows;
  if (bad && threadIdx.x == 0) set_status(a.status, PHS_ERANGE);
  int again = 0;  // the same row listed before: already freed by that entry
  for (int j = threadIdx.x; j < i; j += blockDim.x) again |= a.rows[j] == r;
  if (__syncthreads_or(again) && !bad) {
    if (threadIdx.x == 0) set_status(a.status, PHS_EINVAL);
    bad = 1;
  }
  if (bad) return;
  const int np = held_pages(a.seq_lens[r], a.max_pages, threadIdx.x == 0 ? a.status : nullptr);
  const int32_t* row = a.block_table + static_cast<size_t>(r) * a.max_pages;
  for (int j = threadIdx.x; j < np; j += blockDim.x) {
    const int p = row[j];
    if (p < 0 || p >= a.num_pages) {
      set_status(a.status, PHS_ERANGE);
    } else if (atomicSub(a.refcount + p, 1) <= 0) {  // not live: leave its count as it was
      atomicAdd(a.refcount + p, 1);
      set_status(a.status, PHS_ERANGE);
    }
  }
  __syncthreads();  // every thread has read the length
  if (threadIdx.x == 0) a.seq_lens[r] = 0;
}

int launch_pages_free(const PageFreeArgs& a, cudaStream_t stream) {
  phs_pages_free_kernel<<<a.n, 256, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? PHS_OK : PHS_ECUDA;
}

// Exclusive rank of this thread's `pred` among the CTA's 1024 threads in
// thread order; *total: how many threads have it.
__device__ __forceinline__ int block_rank(bool pred, int* total, int* scratch) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned m = __ballot_sync(0xffffffffu, pred);
  __syncthreads();  // scratch of the previous call is read
  if (lane == 0) scratch[warp] = __popc(m);
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < 32; ++w) {
    const int c = scratch[w];
    if (w < warp) before += c;
    all += c;
  }
  *total = all;
  return before + __popc(m & ((1u << lane) - 1));
}

// ------------------------------------------------------------------ fork --
// Plan: which entries are valid, and the fresh page of each that needs one.
__global__ void __launch_bounds__(1024) phs_pages_fork_plan_kernel(const PageForkArgs a) {
  __shared__ int scratch[32];
  const int tid = threadIdx.x;
  for (int r = tid; r < a.num_rows; r += 1024) {
    a.first_dst[r] = INT32_MAX;
    a.is_src[r] = 0;
  }
  __syncthreads();
  for (int i = tid; i < a.n; i += 1024) {
    const int s = a.src_rows[i], d = a.dst_rows[i];
    if (s >= 0 && s < a.num_rows) a.is_src[s] = 1;
    if (d >= 0 && d < a.num_rows) atomicMin(a.first_dst + d, i);
  }
  __syncthreads();
  int need = 0;  // entries so far that need a fresh page
  for (int base = 0; base < a.n; base += 1024) {
    const int i = base + tid;
    int state = -2, page = -1;
    if (i < a.n) {
      const int s = a.src_rows[i], d = a.dst_rows[i];
      if (s < 0 || s >= a.num_rows || d < 0 || d >= a.num_rows) {
        set_status(a.status, PHS_ERANGE);
      } else if (a.is_src[d] || a.first_dst[d] != i || a.seq_lens[d] != 0) {
        set_status(a.status, PHS_EINVAL);  // the row is not free, or listed twice
      } else {
        const int n = a.seq_lens[s];
        if (n < 0 || n > a.max_pages * kPage) {
          set_status(a.status, PHS_ERANGE);
        } else if (n % kPage == 0) {
          state = -1;
        } else {
          page = a.block_table[static_cast<size_t>(s) * a.max_pages + n / kPage];
          if (page < 0 || page >= a.num_pages || a.refcount[page] <= 0)
            set_status(a.status, PHS_ERANGE);
          else
            state = 0;
        }
      }
    }
    int total;
    const int rank = block_rank(state == 0, &total, scratch);
    if (i < a.n) {
      a.rank[i] = state == 0 ? need + rank : state;
      a.copy_src[i] = page;
    }
    need += total;
  }
  // the lowest `need` free pages
  int found = 0;
  for (int64_t base = 0; base < a.num_pages && found < need; base += 1024) {
    const int64_t p = base + tid;
    int total;
    const bool is_free = p < a.num_pages && a.refcount[p] == 0;
    const int at = found + block_rank(is_free, &total, scratch);
    if (is_free && at < need) a.fresh[at] = static_cast<int32_t>(p);
    found += total;
  }
  __syncthreads();
  for (int i = tid; i < a.n; i += 1024) {
    const int rank = a.rank[i];
    int to = -1;
    if (rank >= 0) {
      if (rank < found) {
        to = a.fresh[rank];
        a.refcount[to] = 1;
      } else {
        set_status(a.status, PHS_ENOSPACE);
        a.rank[i] = -2;
      }
    }
    a.copy_dst[i] = to;
    if (to < 0) a.copy_src[i] = -1;
  }
}

int launch_pages_fork_plan(const PageForkArgs& a, cudaStream_t stream) {
  phs_pages_fork_plan_kernel<<<1, 1024, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? PHS_OK : PHS_ECUDA;
}

// Share: the child's table row, one more reference on each whole page.
__global__ void __launch_bounds__(256) phs_pages_fork_share_kernel(const PageForkArgs a) {
  const int i = blockIdx.x;
  if (a.rank[i] == -2) return;
  const int s = a.src_rows[i], d = a.dst_rows[i], n = a.seq_lens[s];
  const int32_t* from = a.block_table + static_cast<size_t>(s) * a.max_pages;
  int32_t* to = a.block_table + static_cast<size_t>(d) * a.max_pages;
  for (int j = threadIdx.x; j < n / kPage; j += blockDim.x) {
    const int p = from[j];
    to[j] = p;
    if (p < 0 || p >= a.num_pages || a.refcount[p] <= 0)
      set_status(a.status, PHS_ERANGE);
    else
      atomicAdd(a.refcount + p, 1);
  }
  if (threadIdx.x == 0) {
    if (n % kPage != 0) to[n / kPage] = a.copy_dst[i];
    a.seq_lens[d] = n;
  }
}

int launch_pages_fork_share(const PageForkArgs& a, cudaStream_t stream) {
  phs_pages_fork_share_kernel<<<a.n, 256, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? PHS_OK : PHS_ECUDA;
}

// --------------------------------------------------------------- compact --
// Plan: with L live pages in all, the live pages at or above L move, the
// highest first, into the holes below L, the lowest first.
__global__ void __launch_bounds__(1024) phs_pages_compact_plan_kernel(const PageCompactArgs a) {
  __shared__ int scratch[32];
  const int tid = threadIdx.x;
  int live = 0;
  for (int64_t base = 0; base < a.num_pages; base += 1024) {
    const int64_t p = base + tid;
    int total;
    block_rank(p < a.num_pages && a.refcount[p] > 0, &total, scratch);
    live += total;
  }
  int before = 0, moves = 0;
  for (int64_t base = 0; base < a.num_pages; base += 1024) {
    const int64_t p = base + tid;
    const bool in = p < a.num_pages;
    const bool is_live = in && a.refcount[p] > 0;
    int total;
    const int rank = before + block_rank(is_live, &total, scratch);  // live pages below p
    if (in) {
      const int id = static_cast<int32_t>(p);
      if (is_live && id >= live) {
        a.move[p] = live - 1 - rank;
        a.movers[live - 1 - rank] = id;
      } else {
        a.move[p] = is_live ? -2 : -1;
        if (!is_live && id < live) a.holes[id - rank] = id;
      }
    }
    int here;
    block_rank(is_live && p >= live, &here, scratch);
    moves += here;
    before += total;
  }
  if (tid == 0) {
    a.meta[0] = live;
    a.meta[1] = moves;
    *a.num_live = live;
  }
}

int launch_pages_compact_plan(const PageCompactArgs& a, cudaStream_t stream) {
  phs_pages_compact_plan_kernel<<<1, 1024, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? PHS_OK : PHS_ECUDA;
}

// Page map, counts and block tables by the plan.  Every cell is read and
// written by one thread, so the outputs may be the inputs.
__global__ void __launch_bounds__(256) phs_pages_compact_tables_kernel(const PageCompactArgs a) {
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int live = a.meta[0];
  for (int64_t p = t0; p < a.num_pages; p += stride) {
    const int m = a.move[p], count = a.refcount[p];
    if (m >= 0) {
      const int to = a.holes[m];
      a.page_map[p] = to;
      a.refcount_out[to] = count;
      a.refcount_out[p] = 0;
    } else {
      a.page_map[p] = m == -2 ? static_cast<int32_t>(p) : -1;
      if (m == -2 || p >= live) a.refcount_out[p] = count;  // a hole's count is its mover's
    }
  }
  const int64_t cells = static_cast<int64_t>(a.num_rows) * a.max_pages;
  for (int64_t c = t0; c < cells; c += stride) {
    const int r = static_cast<int>(c / a.max_pages), j = static_cast<int>(c % a.max_pages);
    int p = a.block_table[c];
    if (j < held_pages(a.seq_lens[r], a.max_pages, j == 0 ? a.status : nullptr)) {
      const int m = p >= 0 && p < a.num_pages ? a.move[p] : -1;
      if (m >= 0)
        p = a.holes[m];
      else if (m == -1)
        set_status(a.status, PHS_ERANGE);  // not a live page: left as it is
    }
    a.block_table_out[c] = p;
  }
}

int launch_pages_compact_tables(const PageCompactArgs& a, cudaStream_t stream) {
  phs_pages_compact_tables_kernel<<<304, 256, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? PHS_OK : PHS_ECUDA;
}

// ------------------------------------------------------------------ copy --
__global__ void __launch_bounds__(256) phs_pages_copy_kernel(const __grid_constant__ PagePools p,
                                                             const int32_t* src,
                                                             const int32_t* dst,
                                                             const int32_t* n_dev, int64_t n) {
  const int64_t items = (n_dev ? *n_dev : n) * p.num_layers * 2;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t i = it / (2 * p.num_layers);
    const int l = static_cast<int>(it % (2 * p.num_layers));
    if (src[i] < 0) continue;
    uint4* base = l < p.num_layers ? p.k[l] : p.v[l - p.num_layers];
    const uint4* from = base + static_cast<size_t>(src[i]) * p.page_vecs;
    uint4* to = base + static_cast<size_t>(dst[i]) * p.page_vecs;
    for (int e = threadIdx.x; e < p.page_vecs; e += 256) to[e] = from[e];
  }
}

int launch_pages_copy(const PagePools& p, const int32_t* src, const int32_t* dst,
                      const int32_t* n_dev, int64_t n, int num_sms, cudaStream_t stream) {
  phs_pages_copy_kernel<<<num_sms * 8, 256, 0, stream>>>(p, src, dst, n_dev, n);
  return cudaGetLastError() == cudaSuccess ? PHS_OK : PHS_ECUDA;
}

}  // namespace phs
