// phs_pages.cu -- device-side page operations of a paged cache: freeing and
// forking requests and compacting the pool, with the block tables, lengths
// and reference counts that the decode kernels read kept on the device (no
// host round trip, recordable into a graph).
//
// Everything here is integer bookkeeping and byte copies.  Results do not
// depend on the order of atomics: counts are sums, and every choice of a
// page goes by rank in page order (the lowest free pages to the forks in
// their order; the highest live page to the lowest hole).
#include <algorithm>

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
// row's length is zero.  Bound by the latency of two dependent reads and an
// atomic (192 rows of up to 1,024 pages: 9 us, most of it the launch).
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

// A tile is 8 x 1024 consecutive ids on 1024 threads: warp w holds ids
// 256 w .. 256 w + 255 of the tile, thread `lane` its ids 32 k + lane.
constexpr int kTileIds = kPagesTile;
static_assert(kTileIds == 8 * 1024, "tile of 1024 threads");

// Ranks of the marked ids of a tile, in id order.  `mark(k)` says whether this
// thread's k-th id is marked; rank[k] is the number of marked ids of the tile
// before it, the result their number in all.  `scratch`: 64 ints, `turn`
// alternates between calls (one barrier a call).
template <typename Mark>
__device__ __forceinline__ int tile_ranks(Mark&& mark, int (&rank)[8], int* scratch, int turn) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int mine = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const unsigned m = __ballot_sync(0xffffffffu, mark(k));
    rank[k] = mine + __popc(m & ((1u << lane) - 1));
    mine += __popc(m);
  }
  int* sums = scratch + 32 * (turn & 1);
  if (lane == 0) sums[warp] = mine;
  __syncthreads();
  int upto = sums[lane];  // inclusive sums over the warps
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  const int total = __shfl_sync(0xffffffffu, upto, 31);
  const int before = __shfl_sync(0xffffffffu, upto, warp) - mine;
#pragma unroll
  for (int k = 0; k < 8; ++k) rank[k] += before;
  return total;
}
__device__ __forceinline__ int tile_id(int k) {
  return (threadIdx.x >> 5) * 256 + 32 * k + (threadIdx.x & 31);
}

// ------------------------------------------------------------------ copy --
// Pages src[i] -> dst[i], i < n, of every pool (a negative src: none), by
// `ctas` CTAs of 256 threads of which this is number `cta`.  A warp takes
// 2 KB units (every page is a whole number of them: 16 tokens of 64 or 128
// bf16) in turn, 4 16-byte vectors a lane; 64 warps of an SM then have
// 128 KB in flight, which is what the copy needs to run at the memory's rate.
constexpr int kUnitVecs = 128;

__device__ __forceinline__ void copy_pages_by(const PagePools& p, const int32_t* src,
                                              const int32_t* dst, int n, int cta, int ctas) {
  const int lane = threadIdx.x & 31, per_page = p.page_vecs / kUnitVecs, tensors = 2 * p.num_layers;
  const int64_t units = static_cast<int64_t>(n) * tensors * per_page;
  const int64_t step = static_cast<int64_t>(ctas) * 8;
  for (int64_t u = static_cast<int64_t>(cta) * 8 + (threadIdx.x >> 5); u < units; u += step) {
    const int64_t item = u / per_page;
    const int part = static_cast<int>(u - item * per_page);
    const int64_t i = item / tensors;
    const int l = static_cast<int>(item - i * tensors);
    const int from = src[i];
    if (from < 0) continue;
    uint4* base = (l < p.num_layers ? p.k[l] : p.v[l - p.num_layers]) + part * kUnitVecs + lane;
    const uint4* a = base + static_cast<size_t>(from) * p.page_vecs;
    uint4* b = base + static_cast<size_t>(dst[i]) * p.page_vecs;
    uint4 x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = __ldcs(a + 32 * k);
#pragma unroll
    for (int k = 0; k < 4; ++k) __stcs(b + 32 * k, x[k]);
  }
}

// CTAs for copying up to n pages: a warp per unit, at most 8 CTAs an SM
static int64_t copy_ctas(const PagePools& p, int64_t n, int num_sms) {
  const int64_t units = n * 2 * p.num_layers * (p.page_vecs / kUnitVecs);
  return std::max<int64_t>(1, std::min<int64_t>((units + 7) / 8, int64_t{8} * num_sms));
}

// ------------------------------------------------------------------ fork --
// Plan: which entries are valid, and the fresh page of each that needs one, by
// one CTA: the choice of a page depends on all entries before it and on all
// counts, which one CTA reads in a few rounds (12 us for 192 entries of 64
// requests of up to 16,384 tokens, nearly all latency; more CTAs would need
// another launch between the counts and the choice).
__global__ void __launch_bounds__(1024) phs_pages_fork_plan_kernel(const PageForkArgs a) {
  __shared__ int scratch[64];
  const int tid = threadIdx.x;
  pdl_launch_dependents();
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
  int need = 0, turn = 0;  // entries so far that need a fresh page
  for (int base = 0; base < a.n; base += kTileIds) {
    int state[8], rank[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = base + tile_id(k);
      state[k] = -2;
      if (i >= a.n) continue;
      int page = -1;
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
          state[k] = -1;
        } else {
          page = a.block_table[static_cast<size_t>(s) * a.max_pages + n / kPage];
          if (page < 0 || page >= a.num_pages || a.refcount[page] <= 0)
            set_status(a.status, PHS_ERANGE);
          else
            state[k] = 0;
        }
      }
      a.copy_src[i] = page;
    }
    const int total = tile_ranks([&](int k) { return state[k] == 0; }, rank, scratch, turn++);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = base + tile_id(k);
      if (i < a.n) a.rank[i] = state[k] == 0 ? need + rank[k] : state[k];
    }
    need += total;
  }
  // the lowest `need` free pages
  int found = 0;
  for (int64_t base = 0; base < a.num_pages && found < need; base += kTileIds) {
    bool is_free[8];
    int rank[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int64_t p = base + tile_id(k);
      is_free[k] = p < a.num_pages && a.refcount[p] == 0;
    }
    const int total = tile_ranks([&](int k) { return is_free[k]; }, rank, scratch, turn++);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (is_free[k] && found + rank[k] < need)
        a.fresh[found + rank[k]] = static_cast<int32_t>(base + tile_id(k));
    found += total;
  }
  for (int i = min(found, need) + tid; i < a.n; i += 1024) a.fresh[i] = INT32_MAX;
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

// Whether the plan has given out page pg: it then counts 1, as a live page may,
// but an entry that names it named no live page.  (fresh: n ids, ascending.)
__device__ __forceinline__ bool given_out(const int32_t* fresh, int n, int pg) {
  int lo = 0;
  for (int len = n; len > 0;) {
    const int half = len >> 1;
    if (fresh[lo + half] < pg) {
      lo += half + 1;
      len -= half + 1;
    } else {
      len = half;
    }
  }
  return lo < n && fresh[lo] == pg;
}

// Share and copy, side by side in one launch: CTAs [0, n) write a child's
// table row and add a reference on each whole page, the others copy the
// partly filled pages.  192 children, 10 layers, 234 MB read and written: 27 us
// of the copies' 34 at the rate of memory (part of the pages is still in L2).
__global__ void __launch_bounds__(256) phs_pages_fork_kernel(const __grid_constant__ PageForkArgs a,
                                                             const __grid_constant__ PagePools p) {
  pdl_wait_prior_grid();
  if (blockIdx.x >= a.share_ctas) {
    copy_pages_by(p, a.copy_src, a.copy_dst, a.n, blockIdx.x - a.share_ctas,
                  gridDim.x - a.share_ctas);
    return;
  }
  const int i = blockIdx.x;
  if (a.rank[i] == -2) return;
  const int s = a.src_rows[i], d = a.dst_rows[i], n = a.seq_lens[s];
  const int32_t* from = a.block_table + static_cast<size_t>(s) * a.max_pages;
  int32_t* to = a.block_table + static_cast<size_t>(d) * a.max_pages;
  for (int j = threadIdx.x; j < n / kPage; j += blockDim.x) {
    const int pg = from[j];
    to[j] = pg;
    const int count = pg < 0 || pg >= a.num_pages ? 0 : a.refcount[pg];
    if (count <= 0 || (count == 1 && given_out(a.fresh, a.n, pg)))
      set_status(a.status, PHS_ERANGE);
    else
      atomicAdd(a.refcount + pg, 1);
  }
  if (threadIdx.x == 0) {
    if (n % kPage != 0) to[n / kPage] = a.copy_dst[i];
    a.seq_lens[d] = n;
  }
}

// --------------------------------------------------------------- compact --
// With L live pages in all, the live pages at or above L move, the highest
// first, into the holes below L, the lowest first.  Three launches: live
// pages of each tile of ids; the plan, a tile per CTA from the tiles' sums;
// tables and copies.  The first two take a few us each however large the pool
// is; the copies are bound by memory: 3,001 pages moved in 10 layers (3.9 GB
// read and written) take 627 us in all, 6.3 TB/s, against 579 for those bytes at
// the rate of a plain copy; a pool of 512 pages 6.6 us.
__global__ void __launch_bounds__(1024) phs_pages_compact_count_kernel(const PageCompactArgs a) {
  pdl_launch_dependents();
  const int64_t base = static_cast<int64_t>(blockIdx.x) * kTileIds;
  int live = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int64_t p = base + tile_id(k);
    live += __syncthreads_count(p < a.num_pages && a.refcount[p] > 0);
  }
  if (threadIdx.x == 0) a.tile_live[blockIdx.x] = live;
}

__global__ void __launch_bounds__(1024) phs_pages_compact_plan_kernel(const PageCompactArgs a) {
  __shared__ int scratch[64], sums[2];
  const int tid = threadIdx.x, tiles = gridDim.x, tile = blockIdx.x;
  const int64_t base = static_cast<int64_t>(tile) * kTileIds;
  pdl_launch_dependents();
  bool is_live[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int64_t p = base + tile_id(k);
    is_live[k] = p < a.num_pages && a.refcount[p] > 0;
  }
  if (tid < 2) sums[tid] = 0;
  __syncthreads();
  pdl_wait_prior_grid();
  int before = 0, live = 0;
  for (int t = tid; t < tiles; t += 1024) {
    const int c = a.tile_live[t];
    live += c;
    if (t < tile) before += c;
  }
  if (live) atomicAdd(sums, live);
  if (before) atomicAdd(sums + 1, before);
  __syncthreads();
  live = sums[0];
  before = sums[1];
  int rank[8];
  tile_ranks([&](int k) { return is_live[k]; }, rank, scratch, 0);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int64_t p = base + tile_id(k);
    if (p >= a.num_pages) continue;
    const int id = static_cast<int32_t>(p), below = before + rank[k];  // live pages below p
    if (is_live[k] && id >= live) {
      a.move[p] = live - 1 - below;
      a.movers[live - 1 - below] = id;
    } else {
      a.move[p] = is_live[k] ? -2 : -1;
      if (!is_live[k] && id < live) a.holes[id - below] = id;
    }
    if (id == live) a.meta[1] = live - below;  // holes below L = pages that move
  }
  if (tile == 0 && tid == 0) {
    a.meta[0] = live;
    if (live == a.num_pages) a.meta[1] = 0;
    *a.num_live = live;
  }
}

// Page map, counts and block tables by the plan (table_ctas CTAs), and the
// copies (the others).  Every cell is read and written by one thread, so
// the outputs may be the inputs.
__global__ void __launch_bounds__(256)
    phs_pages_compact_kernel(const __grid_constant__ PageCompactArgs a,
                             const __grid_constant__ PagePools p) {
  pdl_wait_prior_grid();
  if (blockIdx.x >= a.table_ctas) {
    copy_pages_by(p, a.movers, a.holes, a.meta[1], blockIdx.x - a.table_ctas,
                  gridDim.x - a.table_ctas);
    return;
  }
  const int64_t stride = static_cast<int64_t>(a.table_ctas) * 256;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int live = a.meta[0];
  for (int64_t pg = t0; pg < a.num_pages; pg += stride) {
    const int m = a.move[pg], count = a.refcount[pg];
    if (m >= 0) {
      const int to = a.holes[m];
      a.page_map[pg] = to;
      a.refcount_out[to] = count;
      a.refcount_out[pg] = 0;
    } else {
      a.page_map[pg] = m == -2 ? static_cast<int32_t>(pg) : -1;
      if (m == -2 || pg >= live) a.refcount_out[pg] = count;  // a hole's count is its mover's
    }
  }
  const int64_t cells = static_cast<int64_t>(a.num_rows) * a.max_pages;
  for (int64_t c = t0; c < cells; c += stride) {
    const int r = static_cast<int>(c / a.max_pages), j = static_cast<int>(c % a.max_pages);
    int pg = a.block_table[c];
    if (j < held_pages(a.seq_lens[r], a.max_pages, j == 0 ? a.status : nullptr)) {
      const int m = pg >= 0 && pg < a.num_pages ? a.move[pg] : -1;
      if (m >= 0)
        pg = a.holes[m];
      else if (m == -1)
        set_status(a.status, PHS_ERANGE);  // not a live page: left as it is
    }
    a.block_table_out[c] = pg;
  }
}

// More pools than one launch takes: their copies alone, by the same plan.
__global__ void __launch_bounds__(256)
    phs_pages_copy_kernel(const __grid_constant__ PagePools p, const int32_t* src,
                          const int32_t* dst, const int32_t* n_dev, int n) {
  copy_pages_by(p, src, dst, n_dev ? *n_dev : n, blockIdx.x, gridDim.x);
}

// ------------------------------------------------------------- launchers --
template <typename... Params, typename... Args>
static int launch_after(void (*kern)(Params...), int64_t grid, int block, cudaStream_t stream,
                        const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(block);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? PHS_OK : PHS_ECUDA;
}

int launch_pages_fork(PageForkArgs a, const PagePools& p, int num_sms, cudaStream_t stream) {
  phs_pages_fork_plan_kernel<<<1, 1024, 0, stream>>>(a);
  if (cudaGetLastError() != cudaSuccess) return PHS_ECUDA;
  a.share_ctas = a.n;
  return launch_after(phs_pages_fork_kernel,
                      int64_t{a.n} + copy_ctas(p, a.n, num_sms), 256, stream, a, p);
}

int launch_pages_compact(PageCompactArgs a, const PagePools& p, int num_sms,
                         cudaStream_t stream) {
  const int64_t tiles = (a.num_pages + kTileIds - 1) / kTileIds;
  phs_pages_compact_count_kernel<<<static_cast<unsigned>(tiles), 1024, 0, stream>>>(a);
  if (cudaGetLastError() != cudaSuccess) return PHS_ECUDA;
  int st = launch_after(phs_pages_compact_plan_kernel, tiles, 1024, stream, a);
  if (st) return st;
  const int64_t cells = std::max(a.num_pages, int64_t{a.num_rows} * a.max_pages);
  a.table_ctas = static_cast<int>(std::min<int64_t>((cells + 255) / 256, num_sms));
  return launch_after(phs_pages_compact_kernel,
                      a.table_ctas + copy_ctas(p, a.num_pages / 2, num_sms), 256, stream, a, p);
}

int launch_pages_copy(const PagePools& p, const int32_t* src, const int32_t* dst,
                      const int32_t* n_dev, int64_t n, int num_sms, cudaStream_t stream) {
  phs_pages_copy_kernel<<<static_cast<unsigned>(copy_ctas(p, n, num_sms)), 256, 0, stream>>>(
      p, src, dst, n_dev, static_cast<int>(n));
  return cudaGetLastError() == cudaSuccess ? PHS_OK : PHS_ECUDA;
}

}  // namespace phs
