// phs_ops.h -- argument blocks and launchers of the page operations
// (phs_pages.cu), differential attention (phs_diff.cu) and linear attention
// (phs_linear.cu), shared with the C-ABI front end (phs_api.cu).
#pragma once

#include "phs_internal.h"

namespace phs {

// ------------------------------------------------------ page operations --
constexpr int kPagesMaxLayers = 64;  // pools per launch

struct PagePools {
  uint4* k[kPagesMaxLayers];
  uint4* v[kPagesMaxLayers];
  int num_layers;
  int page_vecs;  // 16-byte vectors of one page of K (and of V), a multiple of 128
};

struct PageFreeArgs {
  const int32_t* block_table;
  int32_t* seq_lens;
  int32_t* refcount;
  const int32_t* rows;
  int32_t* status;
  int64_t num_pages;
  int num_rows, max_pages, n;
};

struct PageForkArgs {
  int32_t* block_table;
  int32_t* seq_lens;
  int32_t* refcount;
  const int32_t* src_rows;
  const int32_t* dst_rows;
  int32_t* status;
  int64_t num_pages;
  int num_rows, max_pages, n;
  // workspace
  int32_t* first_dst;  // [num_rows] first entry that names the row as its destination
  int32_t* is_src;     // [num_rows]
  int32_t* rank;       // [n] rank among the entries that need a fresh page, -1 none, -2 refused
  int32_t* fresh;      // [n] the pages given out: the lowest free ones, ascending, then INT32_MAX
  int32_t* copy_src;   // [n] page to copy, or -1
  int32_t* copy_dst;   // [n]
  int share_ctas;
};

struct PageCompactArgs {
  const int32_t* block_table;
  int32_t* block_table_out;
  const int32_t* seq_lens;
  const int32_t* refcount;
  int32_t* refcount_out;
  int32_t* page_map;
  int32_t* num_live;
  int32_t* status;
  int64_t num_pages;
  int num_rows, max_pages;
  // workspace
  int32_t* move;    // [num_pages] -1 free, -2 stays, m >= 0: the m-th highest moving page
  int32_t* movers;  // [num_pages] page that is m-th from the top
  int32_t* holes;   // [num_pages] m-th lowest hole
  int32_t* meta;    // [2] live pages, moves
  int32_t* tile_live;  // live pages of each tile of ids
  int table_ctas;
};

constexpr int kPagesTile = 8192;  // ids of a tile

int launch_pages_free(const PageFreeArgs& a, cudaStream_t stream);
int launch_pages_fork(PageForkArgs a, const PagePools& p, int num_sms, cudaStream_t stream);
int launch_pages_compact(PageCompactArgs a, const PagePools& p, int num_sms, cudaStream_t stream);
// pages src[i] -> dst[i] (i < *n_dev, or i < n where n_dev is null; negative
// src: none) of every pool
int launch_pages_copy(const PagePools& p, const int32_t* src, const int32_t* dst,
                      const int32_t* n_dev, int64_t n, int num_sms, cudaStream_t stream);

// ------------------------------------------------ differential attention --
constexpr int kDiffMaxSplit = 4096;  // tokens
constexpr int diff_ctas_per_sm(int D) { return D == 128 ? 1 : 3; }

struct DiffArgs {
  const __nv_bfloat16* q;  // [B][2H][D]
  __nv_bfloat16* k;        // [num_pages][2Hv][16][D]
  __nv_bfloat16* v;
  const __nv_bfloat16* k_new;  // [B][2Hv][D], or null: no append
  const __nv_bfloat16* v_new;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* page_refcount;  // or null
  void* out;               // [B][H][2D]
  float* ws_o;             // [B][Hv][max_splits][G][map][2D]
  float* ws_ml;            // [B][Hv][max_splits][G][map][max, sum]
  int32_t* status;
  int64_t num_pages;
  int H, Hv, G;
  int max_pages;
  int n_clamp;             // lengths above this are an error and clamped
  int T;                   // tokens per split (multiple of 32)
  int max_splits;
  int out_f32;
  float scale_log2;        // softmax_scale * log2(e)
  // weights
  const float* lambda_q1;  // [D], or [H][D] where lambda_per_head
  const float* lambda_k1;
  const float* lambda_q2;
  const float* lambda_k2;
  const float* norm_weight;  // [2D] or null
  float lambda_init, norm_eps;
  int lambda_per_head;
};

int launch_diff_decode(int D, const CUtensorMap& tk, const CUtensorMap& tv, const DiffArgs& a,
                       int B, cudaStream_t stream);

// ------------------------------------------------------ linear attention --
struct LinearArgs {
  const __nv_bfloat16* q;  // [tokens][Hq][D]
  const __nv_bfloat16* k;  // [tokens][Hkv][D]
  const __nv_bfloat16* v;
  float* state;            // [num_states][Hkv][D][D]
  const float* log_decay;  // [Hkv]
  const int32_t* state_ids;  // null: identity
  void* out;               // [tokens][Hq][D]
  int32_t* status;
  int64_t num_states;
  int Hq, Hkv, G, B;
  int out_f32;
  float scale;
  // prompt
  const int32_t* cu_seqlens;  // [B + 1]
  const int32_t* resume;      // [B] or null: from a zero state
  int total_tokens, max_seq;
  int nseg, nsub;             // segments of each prompt, parts of a segment
  int ngrp;                   // CTAs that share a KV head's query heads, a divisor of G
  bool longest_first;         // CTAs in order of their requests' lengths (B <= kLinearSort)
  float* ws;                  // [B][Hkv][nseg * nsub][D][D]: sums of parts, then first states
};

constexpr int kLinearChunk = 128;  // tokens
constexpr int kLinearSort = 256;   // requests of a call that are put in order, at most

int launch_linear_decode(int D, const LinearArgs& a, cudaStream_t stream);
int launch_linear_prompt(int D, const CUtensorMap& tq, const CUtensorMap& tk,
                         const CUtensorMap& tv, const CUtensorMap& to, const LinearArgs& a,
                         cudaStream_t stream);

}  // namespace phs
