// phs_layers.h -- argument blocks and launchers of the rotary cache writes
// (phs_write.cu), the causal convolution (phs_conv.cu) and the selective scan
// (phs_scan.cu), shared with the C-ABI front end (phs_api.cu).
#pragma once

#include "phs_internal.h"

namespace phs {

// ------------------------------------------------------------ cache writes --
struct WriteArgs {
  const __nv_bfloat16* q;  // or null
  const __nv_bfloat16* k;  // or null (phs_rope_rotate of q alone)
  const __nv_bfloat16* v;  // null: phs_rope_rotate
  int64_t q_stride, k_stride, v_stride;  // elements
  __nv_bfloat16* q_out;
  __nv_bfloat16* k_out;  // phs_rope_rotate
  int64_t q_out_stride, k_out_stride;
  const int32_t* positions;   // phs_rope_rotate
  const int32_t* cu_seqlens;  // or null: token b is request b's
  const int32_t* seq_lens;
  const int32_t* block_table;
  const int32_t* page_refcount;  // or null
  int32_t* status;
  __nv_bfloat16* pool_k;
  __nv_bfloat16* pool_v;
  int64_t num_pages;
  int Hq, Hkv, tokens, B, max_pages;
  // rope (rotary 0: none)
  const uint64_t* turns;
  int rotary, interleaved;
  float factor;
  // int8 (codes null: none)
  uint8_t* k_codes;
  uint8_t* v_codes;
  float* k_scale;
  float* v_scale;
  const int32_t* qtable;
  const int32_t* qlens_before;
  const int32_t* qlens;
  int64_t num_qpages;
  int max_qpages, max_qblocks;
  int tile;           // tokens of a CTA
  int q_with_blocks;  // 1: queries of tokens in new blocks are the blocks' launch's
};

struct ReadArgs {
  const __nv_bfloat16* pool_k;
  const __nv_bfloat16* pool_v;
  const int32_t* block_table;
  const int32_t* starts;
  const int32_t* cu_seqlens;
  int32_t* status;
  const uint8_t* k_codes;  // or null
  const uint8_t* v_codes;
  const float* k_scale;
  const float* v_scale;
  const int32_t* qtable;
  const int32_t* qlens;
  __nv_bfloat16* k_out;
  __nv_bfloat16* v_out;
  int64_t num_pages, num_qpages;
  int Hkv, B, tokens, max_tokens, max_pages, max_qpages;
};

constexpr int kWriteMaxTile = 16;  // tokens

int launch_write(int D, WriteArgs a, int num_sms, cudaStream_t stream);
int launch_read_back(int D, const ReadArgs& a, cudaStream_t stream);

// ------------------------------------------------------ causal convolution --
struct ConvArgs {
  const __nv_bfloat16* x;
  int64_t x_stride;
  __nv_bfloat16* state;  // [num_states][width - 1][channels]
  const float* weight;   // [channels][width]
  const float* bias;     // or null
  const int32_t* state_ids;
  const int32_t* cu_seqlens;
  const int32_t* resume;
  __nv_bfloat16* out;
  int32_t* status;
  int64_t num_states;
  int channels, silu, B, tokens;
};

int launch_conv_decode(int width, const ConvArgs& a, cudaStream_t stream);
int launch_conv_prompt(int width, const ConvArgs& a, int num_sms, cudaStream_t stream);

// ---------------------------------------------------------- selective scan --
struct ScanArgs {
  const __nv_bfloat16* x;
  const __nv_bfloat16* b;
  const __nv_bfloat16* c;
  const void* dt;
  int64_t x_stride, b_stride, c_stride, dt_stride;
  int dt_f32;
  float* state;  // [num_states][H][P][N]
  const float* rate;
  const float* skip;     // or null
  const float* dt_bias;  // or null
  const int32_t* state_ids;
  void* out;
  int32_t* status;
  int64_t num_states;
  int H, G, B, out_f32;
  // prompt
  const int32_t* cu_seqlens;
  const int32_t* resume;
  int total_tokens, max_seq;
  int P;
  int slots, units;     // 64 columns of x each, that go together; such units of a request
  int nseg, nsub;       // segments of each prompt, parts of a segment
  int max_chunks;       // of a request
  int short_len;        // requests of up to so many tokens are the short ones' launch's; or -1
  bool longest_first;   // CTAs in order of their requests' lengths (B <= kScanSort)
  float* tables;        // [tokens / 128 + B + 1][H][kScanTable]
  float* ws;            // [B][units][nseg * nsub][64 slots][N]: sums of parts, then first states
  float* ws_log;        // [B][units][nseg * nsub][2]: log decays of the parts
};

constexpr int kScanChunk = 128;  // tokens
constexpr int kScanTable = 536;  // floats
constexpr int kScanShort = 16;   // tokens, at most, that go one by one
constexpr int kScanSort = 256;   // requests of a call that are put in order, at most

int launch_scan_decode(int P, int N, const ScanArgs& a, cudaStream_t stream);
int launch_scan_short(int P, int N, const ScanArgs& a, bool early, cudaStream_t stream);
int launch_scan_prompt(int N, const CUtensorMap& tb, const CUtensorMap& tc, const CUtensorMap& tx,
                       const CUtensorMap& to, const ScanArgs& a, cudaStream_t stream);

}  // namespace phs
