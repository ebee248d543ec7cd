// phs_api.cu -- the extern "C" entry points declared in include/phs.h:
// argument validation, TMA tensor-map encoding, split planning, and the
// hybrid layer-stack driver.  All compute happens in the kernels of
// phs_decode.cu, phs_swa.cu, phs_prefix.cu, phs_append.cu, phs_quant.cu,
// phs_pages.cu, phs_diff.cu, phs_linear.cu, phs_write.cu, phs_conv.cu and phs_scan.cu.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <memory>
#include <map>
#include <mutex>
#include <utility>

#include "phs_internal.h"
#include "phs_layers.h"
#include "phs_ops.h"

namespace phs {

int swa_smem_bytes(int D, int G);

int ensure_dynamic_smem(const void* kernel, int bytes) {
  static std::mutex mu;
  static std::map<std::pair<const void*, int>, int> done;  // (kernel, device) -> bytes set
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PHS_ECUDA;
  std::lock_guard<std::mutex> lock(mu);
  auto it = done.find({kernel, dev});
  if (it != done.end() && it->second >= bytes) return PHS_OK;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) !=
      cudaSuccess)
    return PHS_ECUDA;
  done[{kernel, dev}] = bytes;
  return PHS_OK;
}

namespace {

constexpr int kMaxSplitTokens = 4096;
constexpr int kMaxWindow = 4096;
// The append kernel gives one thread to each 16-byte piece of a token's K
// (and V) row over all KV heads, in one CTA.
constexpr int kMaxAppendThreads = 1024;

// ---------------------------------------------------------- device info --
struct DevInfo {
  int device = -1;
  int sms = 0;
  int smem_optin = 0;
};

int dev_info(DevInfo& out) {
  thread_local DevInfo cache;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PHS_ECUDA;
  if (cache.device != dev) {
    DevInfo d;
    d.device = dev;
    if (cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return PHS_ECUDA;
    if (cudaDeviceGetAttribute(&d.smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) !=
        cudaSuccess)
      return PHS_ECUDA;
    cache = d;
  }
  out = cache;
  return PHS_OK;
}

// ---------------------------------------------------------- tensor maps --
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static std::once_flag once;
  static EncodeTiledFn fn = nullptr;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// bf16 pool viewed as a 2-D tensor of `rows` rows of D elements; boxes of
// 16 rows x 64 columns (128 bytes) with the 128-byte swizzle.
int map_bf16_rows(CUtensorMap* m, const void* base, int64_t rows, int D, uint32_t box_rows = 16) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return PHS_ECUDA;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(D) * 2};
  cuuint32_t box[2] = {64, box_rows};
  cuuint32_t es[2] = {1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides,
                   box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? PHS_OK : PHS_ECUDA;
}

// bf16 pool (D = 128) viewed as a 3-D tensor {64 columns, rows, 2 column
// halves} (strides 256 B, 128 B): one box of {64, 16, 2} fetches a whole
// 16-row page block as [half][16 rows][128 B] with the 128-byte swizzle --
// one 4 KB copy instead of two 2 KB ones (the copy engine's cost is per box).
int map_bf16_pages3d(CUtensorMap* m, const void* base, int64_t rows, uint32_t box_rows = 16) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return PHS_ECUDA;
  cuuint64_t dims[3] = {64, static_cast<cuuint64_t>(rows), 2};
  cuuint64_t strides[2] = {256, 128};
  cuuint32_t box[3] = {64, box_rows, 2};
  cuuint32_t es[3] = {1, 1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides,
                   box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? PHS_OK : PHS_ECUDA;
}

// Map for the per-page K/V copies of the decode kernels: one 3-D box per
// 16-row block when D = 128, two 2-D boxes of 64 columns otherwise (D = 64:
// one box).  Both land as [column half][16 rows][128 B] in shared memory.
// (box_rows 32: two neighbouring heads of a page at once).
int map_bf16_kv(CUtensorMap* m, const void* base, int64_t rows, int D, uint32_t box_rows = 16) {
  return D == 128 ? map_bf16_pages3d(m, base, rows, box_rows)
                  : map_bf16_rows(m, base, rows, D, box_rows);
}

// int8 codes, rows of D bytes; boxes of 32 rows x D with the 128-byte
// (D = 128) or 64-byte (D = 64) swizzle.
int map_i8_rows(CUtensorMap* m, const void* base, int64_t rows, int D) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return PHS_ECUDA;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(D)};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(D), 32};
  cuuint32_t es[2] = {1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box,
                   es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? PHS_OK : PHS_ECUDA;
}

// int8 V^T codes (D x 32 bytes per block and head) viewed as rows of 128
// bytes (4 head dims each); boxes of D/4 rows (a whole block) with the
// 128-byte swizzle: the same copy shape as a K block.
int map_i8_vt(CUtensorMap* m, const void* base, int64_t rows, int D) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return PHS_ECUDA;
  cuuint64_t dims[2] = {128, static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {128};
  cuuint32_t box[2] = {128, static_cast<cuuint32_t>(D / 4)};
  cuuint32_t es[2] = {1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box,
                   es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? PHS_OK : PHS_ECUDA;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_dims(int Hq, int Hkv, int D) {
  if (Hq <= 0 || Hkv <= 0) return PHS_EINVAL;
  if (Hq % Hkv != 0) return PHS_ESHAPE;
  if (Hq / Hkv > 16) return PHS_EUNSUPPORTED;
  if (D != 64 && D != 128) return PHS_EUNSUPPORTED;
  return PHS_OK;
}

int check_paged(const phs_paged_pool* pool) {
  if (!pool || !pool->k || !pool->v) return PHS_EINVAL;
  if (pool->num_pages <= 0 || pool->num_kv_heads <= 0) return PHS_EINVAL;
  if (pool->page_size != kPage) return PHS_EUNSUPPORTED;
  if (pool->head_dim != 64 && pool->head_dim != 128) return PHS_EUNSUPPORTED;
  if (pool->num_pages * pool->num_kv_heads * kPage > INT32_MAX) return PHS_EUNSUPPORTED;
  if (int64_t{pool->num_kv_heads} * pool->head_dim / 8 > kMaxAppendThreads) return PHS_EUNSUPPORTED;
  if (!aligned16(pool->k) || !aligned16(pool->v)) return PHS_EALIGN;
  return PHS_OK;
}

int check_ring(const phs_ring_pool* ring) {
  if (!ring || !ring->k || !ring->v) return PHS_EINVAL;
  if (ring->num_rings <= 0 || ring->num_kv_heads <= 0 || ring->window <= 0) return PHS_EINVAL;
  if (ring->window % kPage != 0 || ring->window > kMaxWindow) return PHS_EUNSUPPORTED;
  if (ring->head_dim != 64 && ring->head_dim != 128) return PHS_EUNSUPPORTED;
  if (ring->num_rings * ring->num_kv_heads * ring->window > INT32_MAX) return PHS_EUNSUPPORTED;
  if (int64_t{ring->num_kv_heads} * ring->head_dim / 8 > kMaxAppendThreads) return PHS_EUNSUPPORTED;
  if (!aligned16(ring->k) || !aligned16(ring->v)) return PHS_EALIGN;
  return PHS_OK;
}

int check_int8(const phs_int8_pool* p) {
  if (!p || !p->k || !p->v || !p->k_scale || !p->v_scale) return PHS_EINVAL;
  if (p->num_qpages <= 0 || p->num_kv_heads <= 0) return PHS_EINVAL;
  if (p->head_dim != 64 && p->head_dim != 128) return PHS_EUNSUPPORTED;
  // TMA row coordinates are int32: 32 K rows and D/4 V^T rows per block and head
  if (p->num_qpages * p->num_kv_heads * kQBlock > INT32_MAX) return PHS_EUNSUPPORTED;
  if (!aligned16(p->k) || !aligned16(p->v)) return PHS_EALIGN;
  return PHS_OK;
}

// Default split length: the longest of 4096, 2048, ... 128 tokens that
// gives the longest request at least 8 splits and whose grid (B x Hkv x
// splits of the longest request) still has 16 CTAs per SM.  Long splits
// amortise each CTA's set-up (queries, page ids, the first copies) and keep
// the partial results small; 8 splits of the longest request keep the last
// wave fine-grained.  Measured (GB/s, whole step, each set on one box; 1024
// / 2048 / 4096 tokens): paged batch 64, lengths to 32K, 7,114 / 7,170 /
// 7,134; INT8 batch 32 at 65K 6,033 / 6,557 / 6,753; 70-layer stack batch
// 256, lengths to 128K, 7,042 / 7,206 / 7,306.
// Short requests in a grid that one wave holds anyway (B x Hkv <= SMs, the
// longest request 129..256 tokens) take one split of 256: no merge then
// follows the decode.  Measured on the 2-layer hybrid step at batch 2
// (lengths 37 and 201, replayed as a CUDA graph): 12.3 -> 10.3 us per step.
#ifndef PHS_SPLIT_T_MAX
#define PHS_SPLIT_T_MAX 4096
#endif
#ifndef PHS_SPLIT_CTAS_PER_SM
#define PHS_SPLIT_CTAS_PER_SM 16
#endif

int32_t plan_tokens_per_split(int B, int Hkv, int max_seq, int requested, int sms) {
  if (requested > 0) return requested;
  if (max_seq > 128 && max_seq <= 256 && static_cast<long long>(B) * Hkv <= sms) return 256;
  int t = PHS_SPLIT_T_MAX;
  while (t > 128 && 8LL * t > max_seq) t /= 2;
  const long long target = static_cast<long long>(PHS_SPLIT_CTAS_PER_SM) * std::max(sms, 1);
  while (t > 128) {
    const long long ctas = static_cast<long long>(B) * Hkv * ((max_seq + t - 1) / t);
    if (ctas >= target) break;
    t /= 2;
  }
  return t;
}

int max_splits_for(int max_seq, int T, bool has_int8) {
  return std::max(1, (max_seq + T - 1) / T + (has_int8 ? 1 : 0));
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

size_t ws_o_bytes(int B, int Hkv, int ms, int G, int D) {
  return align256(static_cast<size_t>(B) * Hkv * ms * G * D * sizeof(float));
}

size_t ws_bytes(int B, int Hkv, int ms, int G, int D) {
  return ws_o_bytes(B, Hkv, ms, G, D) +
         align256(static_cast<size_t>(B) * Hkv * ms * G * 2 * sizeof(float));
}

struct DecodePlan {
  int T = 0, max_splits = 0, G = 0, D = 0, Hkv = 0;
  bool has_int8 = false;
  size_t need = 0;
};

int make_plan(DecodePlan& pl, int B, int Hq, int Hkv, int D, int max_seq, int tps,
              bool has_int8) {
  int st = check_dims(Hq, Hkv, D);
  if (st) return st;
  if (B <= 0 || max_seq < 0) return PHS_EINVAL;
  if (tps < 0 || (tps > 0 && (tps % kQBlock != 0 || tps > kMaxSplitTokens)))
    return PHS_EUNSUPPORTED;
  DevInfo di;
  if ((st = dev_info(di))) return st;
  pl.T = plan_tokens_per_split(B, Hkv, max_seq, tps, di.sms);
  pl.max_splits = max_splits_for(max_seq, pl.T, has_int8);
  pl.G = Hq / Hkv;
  pl.D = D;
  pl.Hkv = Hkv;
  pl.has_int8 = has_int8;
  if (pl.max_splits > 65535) return PHS_EUNSUPPORTED;  // grid z limit
  pl.need = ws_bytes(B, Hkv, pl.max_splits, pl.G, D);
  return PHS_OK;
}

// Shared preamble of the decode entry points.
struct DecodeCall {
  DecodePlan pl;
  SplitArgs a;
  MergeArgs m;
  CUtensorMap tk, tv, tk8, tv8;
};

int prepare_decode(DecodeCall& c, const void* q, int Hq, const phs_paged_pool* pool,
                   const int32_t* block_table, int max_pages, const int32_t* seq_lens,
                   int max_seq, const phs_int8_pool* int8, const int32_t* qtable, int max_qpages,
                   const int32_t* qlens, int B, float softmax_scale, int tps, void* out,
                   int out_dtype, void* workspace, size_t ws_size, const void* k_new,
                   const void* v_new, const int32_t* page_refcount, int32_t* dev_status) {
  int st = check_paged(pool);
  if (st) return st;
  if (!q || !block_table || !seq_lens || !out) return PHS_EINVAL;
  if ((k_new == nullptr) != (v_new == nullptr)) return PHS_EINVAL;
  if (k_new && (!aligned16(k_new) || !aligned16(v_new))) return PHS_EALIGN;
  if (max_pages <= 0 || !(softmax_scale > 0.f) || !std::isfinite(softmax_scale)) return PHS_EINVAL;
  if (out_dtype != PHS_OUT_BF16 && out_dtype != PHS_OUT_F32) return PHS_EINVAL;
  const int D = pool->head_dim, Hkv = pool->num_kv_heads;
  if (int8) {
    if ((st = check_int8(int8))) return st;
    if (!qtable || !qlens || max_qpages <= 0) return PHS_EINVAL;
    if (int8->head_dim != D || int8->num_kv_heads != Hkv) return PHS_ESHAPE;
  }
  if ((st = make_plan(c.pl, B, Hq, Hkv, D, max_seq, tps, int8 != nullptr))) return st;
  if (!workspace || ws_size < c.pl.need) return PHS_EWORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return PHS_EALIGN;
  if (!aligned16(q)) return PHS_EALIGN;

  std::memset(&c.a, 0, sizeof(c.a));
  c.a.q = reinterpret_cast<const __nv_bfloat16*>(q);
  c.a.block_table = block_table;
  c.a.seq_lens = seq_lens;
  c.a.qtable = int8 ? qtable : nullptr;
  c.a.qlens = int8 ? qlens : nullptr;
  c.a.k_scale = int8 ? int8->k_scale : nullptr;
  c.a.v_scale = int8 ? int8->v_scale : nullptr;
  c.a.out = out;
  c.a.ws_o = reinterpret_cast<float*>(workspace);
  c.a.ws_ml = reinterpret_cast<float*>(reinterpret_cast<char*>(workspace) +
                                       ws_o_bytes(B, Hkv, c.pl.max_splits, c.pl.G, D));
  c.a.status = dev_status;
  c.a.num_pages = pool->num_pages;
  c.a.num_qpages = int8 ? int8->num_qpages : 0;
  c.a.Hq = Hq;
  c.a.Hkv = Hkv;
  c.a.G = c.pl.G;
  c.a.max_pages = max_pages;
  c.a.max_qpages = int8 ? max_qpages : 0;
  c.a.n_clamp = static_cast<int>(std::min<long long>(max_seq, 1LL * max_pages * kPage));
  c.a.T = c.pl.T;
  c.a.max_splits = c.pl.max_splits;
  c.a.out_f32 = out_dtype == PHS_OUT_F32;
  c.a.scale_log2 = softmax_scale * 1.4426950408889634f;
  DevInfo di;
  if ((st = dev_info(di))) return st;
  c.a.num_sms = di.sms;
  if (k_new) {  // the step's append, fused into the split launch
    c.a.app = FusedAppend{reinterpret_cast<const __nv_bfloat16*>(k_new),
                          reinterpret_cast<const __nv_bfloat16*>(v_new),
                          reinterpret_cast<__nv_bfloat16*>(pool->k),
                          reinterpret_cast<__nv_bfloat16*>(pool->v)};
    c.a.page_refcount = page_refcount;
  }

  std::memset(&c.m, 0, sizeof(c.m));
  c.m.seq_lens = seq_lens;
  c.m.qlens = c.a.qlens;
  c.m.ws_o = c.a.ws_o;
  c.m.ws_ml = c.a.ws_ml;
  c.m.out = out;
  c.m.Hq = Hq;
  c.m.Hkv = Hkv;
  c.m.G = c.pl.G;
  c.m.n_clamp = c.a.n_clamp;
  c.m.T = c.pl.T;
  c.m.max_splits = c.pl.max_splits;
  c.m.out_f32 = c.a.out_f32;

  const int64_t rows = pool->num_pages * Hkv * kPage;
  if ((st = map_bf16_kv(&c.tk, pool->k, rows, D))) return st;
  if ((st = map_bf16_kv(&c.tv, pool->v, rows, D))) return st;
  if (int8) {
    const int64_t blocks = int8->num_qpages * Hkv;
    if ((st = map_i8_rows(&c.tk8, int8->k, blocks * kQBlock, D))) return st;
    if ((st = map_i8_vt(&c.tv8, int8->v, blocks * (D / 4), D))) return st;
  } else {
    c.tk8 = c.tk;  // unused by bf16-only launches
    c.tv8 = c.tv;
  }
  return PHS_OK;
}

}  // namespace
}  // namespace phs

using namespace phs;

extern "C" {

int32_t phs_version(void) { return 1; }

const char* phs_status_str(int s) {
  switch (s) {
    case PHS_OK: return "ok";
    case PHS_EINVAL: return "invalid argument";
    case PHS_ESHAPE: return "inconsistent shapes";
    case PHS_ERANGE: return "index out of range";
    case PHS_ESHARED: return "append into a shared page";
    case PHS_EWORKSPACE: return "workspace missing or too small";
    case PHS_ECUDA: return "CUDA call failed";
    case PHS_EUNSUPPORTED: return "unsupported shape";
    case PHS_ETIMEOUT: return "device wait timed out";
    case PHS_EALIGN: return "pointer not aligned";
    case PHS_ESCRATCH: return "request exceeds the no-allocation entry point's built-in scratch";
    case PHS_ENOSPACE: return "not enough free pages";
    default: return "unknown status";
  }
}

int phs_kv_append_paged(const phs_paged_pool* pool, const void* k_new, const void* v_new,
                        const int32_t* block_table, int32_t max_pages_per_seq,
                        const int32_t* seq_lens, int32_t batch, const int32_t* page_refcount,
                        int32_t* dev_status, void* stream) {
  int st = check_paged(pool);
  if (st) return st;
  if (!k_new || !v_new || !block_table || !seq_lens || batch < 0 || max_pages_per_seq <= 0)
    return PHS_EINVAL;
  if (!aligned16(k_new) || !aligned16(v_new)) return PHS_EALIGN;
  if (batch == 0) return PHS_OK;
  AppendParams<1> p;
  std::memset(&p, 0, sizeof(p));
  p.layer[0] = AppendLayer{pool->k, pool->v, k_new, v_new, pool->num_pages};
  p.table = block_table;
  p.seq_lens = seq_lens;
  p.refcount = page_refcount;
  p.status = dev_status;
  p.num_layers = 1;
  p.B = batch;
  p.Hkv = pool->num_kv_heads;
  p.D = pool->head_dim;
  p.max_pages = max_pages_per_seq;
  p.is_ring = 0;
  return launch_append<1>(p, reinterpret_cast<cudaStream_t>(stream));
}

int phs_kv_append_ring(const phs_ring_pool* ring, const void* k_new, const void* v_new,
                       const int32_t* ring_ids, const int32_t* ring_pos, int32_t batch,
                       int32_t* dev_status, void* stream) {
  int st = check_ring(ring);
  if (st) return st;
  if (!k_new || !v_new || !ring_pos || batch < 0) return PHS_EINVAL;
  if (!aligned16(k_new) || !aligned16(v_new)) return PHS_EALIGN;
  if (batch == 0) return PHS_OK;
  AppendParams<1> p;
  std::memset(&p, 0, sizeof(p));
  p.layer[0] = AppendLayer{ring->k, ring->v, k_new, v_new, ring->num_rings};
  p.table = ring_ids;
  p.ring_pos = ring_pos;
  p.status = dev_status;
  p.num_layers = 1;
  p.B = batch;
  p.Hkv = ring->num_kv_heads;
  p.D = ring->head_dim;
  p.W = ring->window;
  p.is_ring = 1;
  return launch_append<1>(p, reinterpret_cast<cudaStream_t>(stream));
}

int phs_kv_quant_int8_block32(const phs_paged_pool* src, const int32_t* src_block_table,
                              int32_t src_max_pages, const phs_int8_pool* dst,
                              const int32_t* dst_qtable, int32_t dst_max_qpages,
                              const int32_t* first_qblock, const int32_t* num_qblocks,
                              int32_t max_qblocks, int32_t batch, int32_t* dev_status,
                              void* stream) {
  int st = check_paged(src);
  if (st) return st;
  if ((st = check_int8(dst))) return st;
  if (!src_block_table || !dst_qtable || !first_qblock || !num_qblocks) return PHS_EINVAL;
  if (src_max_pages <= 0 || dst_max_qpages <= 0 || batch < 0 || max_qblocks < 0)
    return PHS_EINVAL;
  if (dst->head_dim != src->head_dim || dst->num_kv_heads != src->num_kv_heads) return PHS_ESHAPE;
  if (batch == 0 || max_qblocks == 0) return PHS_OK;
  QuantArgs a;
  std::memset(&a, 0, sizeof(a));
  a.k_src = reinterpret_cast<const __nv_bfloat16*>(src->k);
  a.v_src = reinterpret_cast<const __nv_bfloat16*>(src->v);
  a.src_table = src_block_table;
  a.k_codes = dst->k;
  a.v_codes = dst->v;
  a.k_scale = dst->k_scale;
  a.v_scale = dst->v_scale;
  a.dst_qtable = dst_qtable;
  a.first_qblock = first_qblock;
  a.num_qblocks = num_qblocks;
  a.status = dev_status;
  a.num_pages = src->num_pages;
  a.num_qpages = dst->num_qpages;
  a.src_max_pages = src_max_pages;
  a.dst_max_qpages = dst_max_qpages;
  a.Hkv = src->num_kv_heads;
  a.D = src->head_dim;
  return launch_quant(a, max_qblocks, batch, reinterpret_cast<cudaStream_t>(stream));
}

int32_t phs_decode_tokens_per_split(int32_t batch, int32_t num_kv_heads, int32_t max_seq_len,
                                    int32_t tokens_per_split) {
  DevInfo di;
  if (dev_info(di)) return PHS_ECUDA;
  if (tokens_per_split < 0 || (tokens_per_split > 0 && (tokens_per_split % kQBlock != 0 ||
                                                        tokens_per_split > kMaxSplitTokens)))
    return PHS_EUNSUPPORTED;
  return plan_tokens_per_split(batch, num_kv_heads, max_seq_len, tokens_per_split, di.sms);
}

size_t phs_decode_workspace_bytes(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                                  int32_t head_dim, int32_t max_seq_len,
                                  int32_t tokens_per_split, int32_t has_int8) {
  DecodePlan pl;
  if (make_plan(pl, batch, num_q_heads, num_kv_heads, head_dim, max_seq_len, tokens_per_split,
                has_int8 != 0))
    return 0;
  return pl.need;
}

int phs_attn_decode_full_paged_split(const void* q, int32_t num_q_heads,
                                     const phs_paged_pool* pool, const int32_t* block_table,
                                     int32_t max_pages_per_seq, const int32_t* seq_lens,
                                     int32_t max_seq_len, const phs_int8_pool* int8,
                                     const int32_t* qtable, int32_t max_qpages_per_seq,
                                     const int32_t* qlens, int32_t batch, float softmax_scale,
                                     int32_t tokens_per_split, void* out, int32_t out_dtype,
                                     void* workspace, size_t workspace_bytes, const void* k_new,
                                     const void* v_new, const int32_t* page_refcount,
                                     int32_t* dev_status, void* stream) {
  DecodeCall c;
  int st = prepare_decode(c, q, num_q_heads, pool, block_table, max_pages_per_seq, seq_lens,
                          max_seq_len, int8, qtable, max_qpages_per_seq, qlens, batch,
                          softmax_scale, tokens_per_split, out, out_dtype, workspace,
                          workspace_bytes, k_new, v_new, page_refcount, dev_status);
  if (st) return st;
  return launch_split_decode(c.pl.D, c.tk, c.tv, c.tk8, c.tv8, c.a, batch,
                             reinterpret_cast<cudaStream_t>(stream));
}

int phs_attn_merge_splits(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                          int32_t head_dim, const int32_t* seq_lens, int32_t max_seq_len,
                          const int32_t* qlens, int32_t has_int8, int32_t tokens_per_split,
                          void* out, int32_t out_dtype, const void* workspace,
                          size_t workspace_bytes, void* stream) {
  DecodePlan pl;
  int st = make_plan(pl, batch, num_q_heads, num_kv_heads, head_dim, max_seq_len,
                     tokens_per_split, has_int8 != 0);
  if (st) return st;
  if (!seq_lens || !out) return PHS_EINVAL;
  if (has_int8 && !qlens) return PHS_EINVAL;
  if (out_dtype != PHS_OUT_BF16 && out_dtype != PHS_OUT_F32) return PHS_EINVAL;
  if (!workspace || workspace_bytes < pl.need) return PHS_EWORKSPACE;
  MergeArgs m;
  std::memset(&m, 0, sizeof(m));
  m.seq_lens = seq_lens;
  m.qlens = has_int8 ? qlens : nullptr;
  m.ws_o = reinterpret_cast<const float*>(workspace);
  m.ws_ml = reinterpret_cast<const float*>(reinterpret_cast<const char*>(workspace) +
                                           ws_o_bytes(batch, num_kv_heads, pl.max_splits, pl.G,
                                                      head_dim));
  m.out = out;
  m.Hq = num_q_heads;
  m.Hkv = num_kv_heads;
  m.G = pl.G;
  m.n_clamp = max_seq_len;
  m.T = pl.T;
  m.max_splits = pl.max_splits;
  m.out_f32 = out_dtype == PHS_OUT_F32;
  return launch_merge(head_dim, m, batch, reinterpret_cast<cudaStream_t>(stream));
}

namespace {

// The decode call; allow_wide = false keeps 4 warps per CTA whatever the
// grid (the unfused stack decides for the whole step, as the fused one does).
int decode_full_paged(const void* q, int32_t num_q_heads, const phs_paged_pool* pool,
                      const int32_t* block_table, int32_t max_pages_per_seq,
                      const int32_t* seq_lens, int32_t max_seq_len, const phs_int8_pool* int8,
                      const int32_t* qtable, int32_t max_qpages_per_seq, const int32_t* qlens,
                      int32_t batch, float softmax_scale, int32_t tokens_per_split, void* out,
                      int32_t out_dtype, void* workspace, size_t workspace_bytes,
                      const void* k_new, const void* v_new, const int32_t* page_refcount,
                      int32_t* dev_status, void* stream, bool allow_wide) {
  DecodeCall c;
  int st = prepare_decode(c, q, num_q_heads, pool, block_table, max_pages_per_seq, seq_lens,
                          max_seq_len, int8, qtable, max_qpages_per_seq, qlens, batch,
                          softmax_scale, tokens_per_split, out, out_dtype, workspace,
                          workspace_bytes, k_new, v_new, page_refcount, dev_status);
  if (st) return st;
  if (!allow_wide) c.a.num_sms = 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if ((st = launch_split_decode(c.pl.D, c.tk, c.tv, c.tk8, c.tv8, c.a, batch, s))) return st;
  if (c.pl.max_splits == 1) return PHS_OK;  // every request finished in its only split
  return launch_merge(c.pl.D, c.m, batch, s);
}

}  // namespace

int phs_attn_decode_full_paged(const void* q, int32_t num_q_heads, const phs_paged_pool* pool,
                               const int32_t* block_table, int32_t max_pages_per_seq,
                               const int32_t* seq_lens, int32_t max_seq_len,
                               const phs_int8_pool* int8, const int32_t* qtable,
                               int32_t max_qpages_per_seq, const int32_t* qlens, int32_t batch,
                               float softmax_scale, int32_t tokens_per_split, void* out,
                               int32_t out_dtype, void* workspace, size_t workspace_bytes,
                               const void* k_new, const void* v_new,
                               const int32_t* page_refcount, int32_t* dev_status, void* stream) {
  return decode_full_paged(q, num_q_heads, pool, block_table, max_pages_per_seq, seq_lens,
                           max_seq_len, int8, qtable, max_qpages_per_seq, qlens, batch,
                           softmax_scale, tokens_per_split, out, out_dtype, workspace,
                           workspace_bytes, k_new, v_new, page_refcount, dev_status, stream, true);
}

int phs_attn_decode_swa_ring(const void* q, int32_t num_q_heads, const phs_ring_pool* ring,
                             const int32_t* ring_ids, const int32_t* ring_pos,
                             const int32_t* seq_lens, int32_t batch, float softmax_scale,
                             void* out, int32_t out_dtype, int32_t* dev_status, void* stream) {
  int st = check_ring(ring);
  if (st) return st;
  if (!q || !ring_pos || !seq_lens || !out || batch < 0) return PHS_EINVAL;
  if (!(softmax_scale > 0.f) || !std::isfinite(softmax_scale)) return PHS_EINVAL;
  if (out_dtype != PHS_OUT_BF16 && out_dtype != PHS_OUT_F32) return PHS_EINVAL;
  const int D = ring->head_dim, Hkv = ring->num_kv_heads;
  if ((st = check_dims(num_q_heads, Hkv, D))) return st;
  if (!aligned16(q)) return PHS_EALIGN;
  if (batch == 0) return PHS_OK;
  DevInfo di;
  if ((st = dev_info(di))) return st;
  if (swa_smem_bytes(D, num_q_heads / Hkv) > di.smem_optin) return PHS_EUNSUPPORTED;
  SwaParams<1> p;
  std::memset(&p, 0, sizeof(p));
  if ((st = map_bf16_kv(&p.tk[0], ring->k, ring->num_rings * Hkv * ring->window, D))) return st;
  if ((st = map_bf16_kv(&p.tv[0], ring->v, ring->num_rings * Hkv * ring->window, D))) return st;
  p.q[0] = reinterpret_cast<const __nv_bfloat16*>(q);
  p.out[0] = out;
  p.num_rings[0] = ring->num_rings;
  p.ring_ids = ring_ids;
  p.ring_pos = ring_pos;
  p.seq_lens = seq_lens;
  p.status = dev_status;
  p.num_layers = 1;
  p.B = batch;
  p.Hq = num_q_heads;
  p.Hkv = Hkv;
  p.G = num_q_heads / Hkv;
  p.W = ring->window;
  p.out_f32 = out_dtype == PHS_OUT_F32;
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  return launch_swa_decode<1>(D, p, di.sms, di.smem_optin, reinterpret_cast<cudaStream_t>(stream));
}

// ------------------------------------------------- shared-prefix decode --
namespace {

struct PrefixPlan {
  int G = 0, rows = 0, T = 0, ms = 0, ntiles = 0, tps = 0, nsp = 0;
  size_t off_ml = 0, off_po = 0, off_pml = 0, off_bad = 0, need = 0;
};

int make_prefix_plan(PrefixPlan& pl, int B, int Hq, int Hkv, int D, int max_seq, int shared_len) {
  int st = check_dims(Hq, Hkv, D);
  if (st) return st;
  if (D != 128) return PHS_EUNSUPPORTED;
  if (B <= 0 || shared_len <= 0 || max_seq < shared_len) return PHS_EINVAL;
  if (shared_len % 64 != 0) return PHS_EUNSUPPORTED;
  pl.G = Hq / Hkv;
  pl.rows = B * pl.G;
  if (pl.rows > 256) return PHS_EUNSUPPORTED;
  DevInfo di;
  if ((st = dev_info(di))) return st;
  if (prefix_smem_bytes() > di.smem_optin) return PHS_EUNSUPPORTED;
  const int suffix = std::max(1, max_seq - shared_len);
  // own-token splits of at least 256 tokens: they run beside the prefix pass
  // on the spare SMs, where fewer and longer CTAs spend less on set-up per
  // byte (250,000-token prefix, 64 requests with 512-640 own tokens: 128 ->
  // 256 tokens per split took the call from 0.2300 to 0.2270-0.2275 ms)
  pl.T = std::max(256, plan_tokens_per_split(B, Hkv, suffix, 0, di.sms));
  pl.ms = std::max(1, (suffix + pl.T - 1) / pl.T);
  pl.ntiles = shared_len / 64;
  // One CTA per SM: each KV head's prefix is spread over (SMs - spare) / Hkv
  // CTAs.  The spare SMs run the own-token split while the prefix pass runs
  // (its CTAs cannot share an SM with a prefix CTA; without spare SMs they
  // all run in the pass's tail).  spare balances the two: own tokens at the
  // split kernel's rate against prefix tokens at the prefix pass's (about
  // 48 and 32 GB/s per SM), over the longest own suffix.  Measured on the
  // 250,000-token prefix, 64 requests (decode call): 0 spare SMs 0.2405 ms,
  // 8 0.2381, 16 0.2349, 24 0.2375; this rule gives 16 there.
  const double own = static_cast<double>(B) * std::max(0, max_seq - shared_len);
  const double share = own / (own + 1.5 * static_cast<double>(shared_len));
  const int spare = std::min(di.sms / 2, static_cast<int>(share * di.sms + 0.5));
  const int target = std::max(1, (di.sms - spare) / Hkv);
  pl.tps = (pl.ntiles + target - 1) / target;
  pl.nsp = (pl.ntiles + pl.tps - 1) / pl.tps;
  if (pl.nsp > 65535) return PHS_EUNSUPPORTED;
  pl.off_ml = ws_o_bytes(B, Hkv, pl.ms, pl.G, D);
  pl.off_po = pl.off_ml + align256(static_cast<size_t>(B) * Hkv * pl.ms * pl.G * 2 * sizeof(float));
  pl.off_pml = pl.off_po + align256(static_cast<size_t>(Hkv) * pl.nsp * 256 * D * sizeof(float));
  pl.off_bad = pl.off_pml + align256(static_cast<size_t>(Hkv) * pl.nsp * 256 * 2 * sizeof(float));
  pl.need = pl.off_bad + align256(static_cast<size_t>(B) * Hkv * pl.ms * sizeof(int32_t));
  return PHS_OK;
}

}  // namespace

size_t phs_shared_prefix_workspace_bytes(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                                         int32_t head_dim, int32_t max_seq_len,
                                         int32_t shared_len) {
  PrefixPlan pl;
  if (make_prefix_plan(pl, batch, num_q_heads, num_kv_heads, head_dim, max_seq_len, shared_len))
    return 0;
  return pl.need;
}

int phs_attn_decode_shared_prefix(const void* q, int32_t num_q_heads, const phs_paged_pool* pool,
                                  const int32_t* block_table, int32_t max_pages_per_seq,
                                  const int32_t* seq_lens, int32_t max_seq_len, int32_t batch,
                                  int32_t shared_len, float softmax_scale, void* out,
                                  int32_t out_dtype, void* workspace, size_t workspace_bytes,
                                  const void* k_new, const void* v_new,
                                  const int32_t* page_refcount, int32_t* dev_status,
                                  void* stream) {
  int st = check_paged(pool);
  if (st) return st;
  if (!q || !block_table || !seq_lens || !out) return PHS_EINVAL;
  if ((k_new == nullptr) != (v_new == nullptr)) return PHS_EINVAL;
  if (k_new && (!aligned16(k_new) || !aligned16(v_new))) return PHS_EALIGN;
  if (max_pages_per_seq <= 0 || !(softmax_scale > 0.f) || !std::isfinite(softmax_scale))
    return PHS_EINVAL;
  if (out_dtype != PHS_OUT_BF16 && out_dtype != PHS_OUT_F32) return PHS_EINVAL;
  const int D = pool->head_dim, Hkv = pool->num_kv_heads;
  PrefixPlan pl;
  if ((st = make_prefix_plan(pl, batch, num_q_heads, Hkv, D, max_seq_len, shared_len))) return st;
  if (shared_len / kPage > max_pages_per_seq) return PHS_ESHAPE;
  if (!workspace || workspace_bytes < pl.need) return PHS_EWORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || !aligned16(q)) return PHS_EALIGN;
  char* ws = reinterpret_cast<char*>(workspace);
  CUtensorMap tk;  // 64-column boxes: the prefix kernel's K tile is [half][64 rows]
  const int64_t rows = pool->num_pages * Hkv * kPage;
  if ((st = map_bf16_rows(&tk, pool->k, rows, D))) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const float scale_log2 = softmax_scale * 1.4426950408889634f;
  // 1. the shared prefix, all requests at once (tensor cores)
  PrefixArgs pa;
  std::memset(&pa, 0, sizeof(pa));
  pa.q = reinterpret_cast<const __nv_bfloat16*>(q);
  pa.block_table = block_table;  // row 0 holds the shared prefix pages
  pa.status = dev_status;
  pa.ws_o = reinterpret_cast<float*>(ws + pl.off_po);
  pa.ws_ml = reinterpret_cast<float*>(ws + pl.off_pml);
  pa.num_pages = pool->num_pages;
  pa.Hq = num_q_heads;
  pa.Hkv = Hkv;
  pa.G = pl.G;
  pa.rows = pl.rows;
  pa.shared_len = shared_len;
  pa.tiles_per_split = pl.tps;
  pa.num_splits = pl.nsp;
  pa.scale_log2 = scale_log2;
  CUtensorMap tk3, tv3;  // per-page boxes (split kernel K/V, prefix kernel V)
  if ((st = map_bf16_pages3d(&tk3, pool->k, rows))) return st;
  if ((st = map_bf16_pages3d(&tv3, pool->v, rows))) return st;
  if ((st = launch_prefix_decode(tk, tv3, pa, s))) return st;
  // 2. each request's own tokens [shared_len, n) (split-KV, partials only)
  SplitArgs a;
  std::memset(&a, 0, sizeof(a));
  a.q = pa.q;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.out = out;
  a.ws_o = reinterpret_cast<float*>(ws);
  a.ws_ml = reinterpret_cast<float*>(ws + pl.off_ml);
  a.status = dev_status;
  a.num_pages = pool->num_pages;
  a.Hq = num_q_heads;
  a.Hkv = Hkv;
  a.G = pl.G;
  a.max_pages = max_pages_per_seq;
  a.n_clamp = static_cast<int>(std::min<long long>(max_seq_len, 1LL * max_pages_per_seq * kPage));
  a.T = pl.T;
  a.max_splits = pl.ms;
  a.out_f32 = out_dtype == PHS_OUT_F32;
  a.scale_log2 = scale_log2;
  a.skip_len = shared_len;
  a.force_partial = 1;
  a.prefix_bad = reinterpret_cast<int32_t*>(ws + pl.off_bad);
  a.wait_prior_at_exit = 1;  // started beside the prefix pass (independent tokens)
  if (k_new) {  // the new tokens are own tokens: the own-token split appends them
    a.app = FusedAppend{reinterpret_cast<const __nv_bfloat16*>(k_new),
                        reinterpret_cast<const __nv_bfloat16*>(v_new),
                        reinterpret_cast<__nv_bfloat16*>(pool->k),
                        reinterpret_cast<__nv_bfloat16*>(pool->v)};
    a.page_refcount = page_refcount;
  }
  if ((st = launch_split_decode(D, tk3, tv3, tk3, tv3, a, batch, s, true))) return st;
  // 3. merge prefix and suffix partials
  PrefixMergeArgs m;
  std::memset(&m, 0, sizeof(m));
  m.seq_lens = seq_lens;
  m.prefix_bad = a.prefix_bad;
  m.bad_slots = Hkv * pl.ms;
  m.ws_o = a.ws_o;
  m.ws_ml = a.ws_ml;
  m.ws_po = pa.ws_o;
  m.ws_pml = pa.ws_ml;
  m.out = out;
  m.Hq = num_q_heads;
  m.Hkv = Hkv;
  m.G = pl.G;
  m.n_clamp = a.n_clamp;
  m.T = pl.T;
  m.max_splits = pl.ms;
  m.num_psplits = pl.nsp;
  m.shared_len = shared_len;
  m.out_f32 = a.out_f32;
  return launch_merge_prefix(m, batch, s);
}

size_t phs_hybrid_stack_workspace_bytes(int32_t batch, int32_t num_q_heads,
                                        int32_t num_kv_heads, int32_t head_dim,
                                        int32_t max_seq_len) {
  return phs_decode_workspace_bytes(batch, num_q_heads, num_kv_heads, head_dim, max_seq_len, 0, 0);
}

int phs_attn_decode_hybrid_stack(const phs_layer* layers, int32_t num_layers,
                                 int32_t num_q_heads, int32_t batch, const int32_t* block_table,
                                 int32_t max_pages_per_seq, const int32_t* page_refcount,
                                 const int32_t* seq_lens, int32_t max_seq_len,
                                 const int32_t* ring_ids, const int32_t* ring_pos,
                                 float softmax_scale, int32_t do_append, int32_t out_dtype,
                                 void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                 void* stream) {
  if (!layers || num_layers <= 0 || batch < 0 || !seq_lens) return PHS_EINVAL;
  if (out_dtype != PHS_OUT_BF16 && out_dtype != PHS_OUT_F32) return PHS_EINVAL;
  if (!(softmax_scale > 0.f) || !std::isfinite(softmax_scale)) return PHS_EINVAL;
  if (batch == 0) return PHS_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int st;
  // ---- validate every layer before launching anything
  int D = -1, Hkv = -1, W = -1;
  int nfull = 0, nswa = 0;
  for (int i = 0; i < num_layers; ++i) {
    const phs_layer& L = layers[i];
    if (!L.q || !L.out) return PHS_EINVAL;
    if (do_append && (!L.k_new || !L.v_new)) return PHS_EINVAL;
    int d, h;
    if (L.is_full) {
      if ((st = check_paged(&L.paged))) return st;
      d = L.paged.head_dim;
      h = L.paged.num_kv_heads;
      ++nfull;
    } else {
      if ((st = check_ring(&L.ring))) return st;
      d = L.ring.head_dim;
      h = L.ring.num_kv_heads;
      if (W < 0) W = L.ring.window;
      if (L.ring.window != W) return PHS_ESHAPE;
      ++nswa;
    }
    if (D < 0) {
      D = d;
      Hkv = h;
    }
    if (d != D || h != Hkv) return PHS_ESHAPE;
    if (!aligned16(L.q) || (do_append && (!aligned16(L.k_new) || !aligned16(L.v_new))))
      return PHS_EALIGN;
  }
  if ((st = check_dims(num_q_heads, Hkv, D))) return st;
  if (nfull && (!block_table || max_pages_per_seq <= 0)) return PHS_EINVAL;
  if (nswa && !ring_pos) return PHS_EINVAL;
  DevInfo di;
  if ((st = dev_info(di))) return st;
  if (nswa && swa_smem_bytes(D, num_q_heads / Hkv) > di.smem_optin) return PHS_EUNSUPPORTED;
  // 8 warps per split CTA only if all Full layers' grids together fit one
  // wave (the fused call's launch shape, so both give the same results)
  bool wide = false;
  if (nfull) {
    DecodePlan pl;
    if ((st = make_plan(pl, batch, num_q_heads, Hkv, D, max_seq_len, 0, false))) return st;
    if (!workspace || workspace_bytes < pl.need) return PHS_EWORKSPACE;
    wide = 1LL * batch * Hkv * pl.max_splits * nfull <= di.sms;
  }

  // ---- appends: all Full layers in one launch, all SWA layers in one
  if (do_append) {
    for (int pass = 0; pass < 2; ++pass) {
      const bool full = pass == 0;
      AppendParams<kAppendMaxLayers> p;
      std::memset(&p, 0, sizeof(p));
      p.table = full ? block_table : ring_ids;
      p.seq_lens = seq_lens;
      p.ring_pos = ring_pos;
      p.refcount = full ? page_refcount : nullptr;
      p.status = dev_status;
      p.B = batch;
      p.Hkv = Hkv;
      p.D = D;
      p.max_pages = max_pages_per_seq;
      p.W = W;
      p.is_ring = full ? 0 : 1;
      for (int i = 0; i < num_layers; ++i) {
        const phs_layer& L = layers[i];
        if ((L.is_full != 0) != full) continue;
        p.layer[p.num_layers++] =
            full ? AppendLayer{L.paged.k, L.paged.v, L.k_new, L.v_new, L.paged.num_pages}
                 : AppendLayer{L.ring.k, L.ring.v, L.k_new, L.v_new, L.ring.num_rings};
        if (p.num_layers == kAppendMaxLayers) {
          if ((st = launch_append<kAppendMaxLayers>(p, s))) return st;
          p.num_layers = 0;
        }
      }
      if (p.num_layers && (st = launch_append<kAppendMaxLayers>(p, s))) return st;
    }
  }

  // ---- SWA layers: one launch (per 64 layers)
  if (nswa) {
    SwaParams<kSwaMaxLayers>* p = new SwaParams<kSwaMaxLayers>();
    std::memset(p, 0, sizeof(*p));
    p->ring_ids = ring_ids;
    p->ring_pos = ring_pos;
    p->seq_lens = seq_lens;
    p->status = dev_status;
    p->B = batch;
    p->Hq = num_q_heads;
    p->Hkv = Hkv;
    p->G = num_q_heads / Hkv;
    p->W = W;
    p->out_f32 = out_dtype == PHS_OUT_F32;
    p->scale_log2 = softmax_scale * 1.4426950408889634f;
    st = PHS_OK;
    for (int i = 0; i < num_layers && st == PHS_OK; ++i) {
      const phs_layer& L = layers[i];
      if (L.is_full) continue;
      const int k = p->num_layers;
      const int64_t rows = L.ring.num_rings * Hkv * W;
      if ((st = map_bf16_kv(&p->tk[k], L.ring.k, rows, D))) break;
      if ((st = map_bf16_kv(&p->tv[k], L.ring.v, rows, D))) break;
      p->q[k] = reinterpret_cast<const __nv_bfloat16*>(L.q);
      p->out[k] = L.out;
      p->num_rings[k] = L.ring.num_rings;
      if (++p->num_layers == kSwaMaxLayers) {
        st = launch_swa_decode<kSwaMaxLayers>(D, *p, di.sms, di.smem_optin, s);
        p->num_layers = 0;
      }
    }
    if (st == PHS_OK && p->num_layers) st = launch_swa_decode<kSwaMaxLayers>(D, *p, di.sms, di.smem_optin, s);
    delete p;
    if (st) return st;
  }

  // ---- Full layers: split + merge per layer, reusing the workspace
  for (int i = 0; i < num_layers; ++i) {
    const phs_layer& L = layers[i];
    if (!L.is_full) continue;
    st = decode_full_paged(L.q, num_q_heads, &L.paged, block_table, max_pages_per_seq, seq_lens,
                           max_seq_len, nullptr, nullptr, 0, nullptr, batch, softmax_scale, 0,
                           L.out, out_dtype, workspace, workspace_bytes, nullptr, nullptr, nullptr,
                           dev_status, stream, wide);
    if (st) return st;
  }
  return PHS_OK;
}

size_t phs_hybrid_stack_fused_workspace_bytes(int32_t batch, int32_t num_q_heads,
                                              int32_t num_kv_heads, int32_t head_dim,
                                              int32_t max_seq_len, int32_t num_full_layers) {
  if (num_full_layers <= 0) return 0;
  const size_t one =
      phs_decode_workspace_bytes(batch, num_q_heads, num_kv_heads, head_dim, max_seq_len, 0, 0);
  return one * static_cast<size_t>(num_full_layers);
}

int phs_attn_decode_hybrid_stack_fused(const phs_layer* layers, int32_t num_layers,
                                       int32_t num_q_heads, int32_t batch,
                                       const int32_t* block_table, int32_t max_pages_per_seq,
                                       const int32_t* page_refcount,
                                       const int32_t* seq_lens, int32_t max_seq_len,
                                       const int32_t* ring_ids, const int32_t* ring_pos,
                                       float softmax_scale, int32_t out_dtype, void* workspace,
                                       size_t workspace_bytes, int32_t* dev_status,
                                       void* stream) {
  if (!layers || num_layers <= 0 || batch < 0 || !seq_lens) return PHS_EINVAL;
  if (out_dtype != PHS_OUT_BF16 && out_dtype != PHS_OUT_F32) return PHS_EINVAL;
  if (!(softmax_scale > 0.f) || !std::isfinite(softmax_scale)) return PHS_EINVAL;
  if (batch == 0) return PHS_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int st;
  // ---- validate every layer before launching anything
  int D = -1, Hkv = -1, W = -1, nfull = 0, nswa = 0;
  int64_t min_pages = 0;  // the Full pools share the block table: ids must fit all of them
  for (int i = 0; i < num_layers; ++i) {
    const phs_layer& L = layers[i];
    if (!L.q || !L.out || !L.k_new || !L.v_new) return PHS_EINVAL;
    int d, h;
    if (L.is_full) {
      if ((st = check_paged(&L.paged))) return st;
      d = L.paged.head_dim;
      h = L.paged.num_kv_heads;
      min_pages = nfull == 0 ? L.paged.num_pages : std::min(min_pages, L.paged.num_pages);
      ++nfull;
    } else {
      if ((st = check_ring(&L.ring))) return st;
      d = L.ring.head_dim;
      h = L.ring.num_kv_heads;
      if (W < 0) W = L.ring.window;
      if (L.ring.window != W) return PHS_ESHAPE;
      ++nswa;
    }
    if (D < 0) {
      D = d;
      Hkv = h;
    }
    if (d != D || h != Hkv) return PHS_ESHAPE;
    if (!aligned16(L.q) || !aligned16(L.k_new) || !aligned16(L.v_new)) return PHS_EALIGN;
  }
  if ((st = check_dims(num_q_heads, Hkv, D))) return st;
  if (nfull && (!block_table || max_pages_per_seq <= 0)) return PHS_EINVAL;
  if (nswa && !ring_pos) return PHS_EINVAL;
  DevInfo di;
  if ((st = dev_info(di))) return st;
  if (nswa && swa_smem_bytes(D, num_q_heads / Hkv) > di.smem_optin) return PHS_EUNSUPPORTED;
  DecodePlan pl;
  if (nfull) {
    if ((st = make_plan(pl, batch, num_q_heads, Hkv, D, max_seq_len, 0, false))) return st;
    if (!workspace || workspace_bytes < pl.need * static_cast<size_t>(nfull))
      return PHS_EWORKSPACE;
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return PHS_EALIGN;
  }
  const float scale_log2 = softmax_scale * 1.4426950408889634f;
  StackMergeParams fold_merges;  // Full-layer merges handed to the SWA launch
  std::memset(&fold_merges, 0, sizeof(fold_merges));
  int fold_layers = 0;

  // A small step (every request in one split, so nothing to merge, and the
  // Full CTAs and SWA units together in one wave) goes in one launch that
  // runs both kinds of layer (phs_stack_small_kernel); the parameter blocks
  // below are built as for the two launches and handed to it.
  std::unique_ptr<StackSmallParams> small;
  if (nfull && nswa && nfull < kStackMaxFull && nswa < kSwaMaxLayers && pl.max_splits == 1 &&
      1LL * batch * Hkv * (nfull + nswa) <= di.sms &&
      stack_small_smem_bytes(D, num_q_heads / Hkv, di.smem_optin) > 0) {
    small.reset(new StackSmallParams());
    std::memset(small.get(), 0, sizeof(StackSmallParams));
  }

  // ---- launch 1 (per 16 Full layers): split-KV decode of every Full layer,
  // each CTA holding a request's newest token also appends it
  if (nfull) {
    StackFullParams* p = new StackFullParams();
    std::memset(p, 0, sizeof(*p));
    StackMergeParams* m = new StackMergeParams();
    std::memset(m, 0, sizeof(*m));
    SplitArgs& a = p->a;
    a.block_table = block_table;
    a.page_refcount = page_refcount;
    a.seq_lens = seq_lens;
    a.status = dev_status;
    a.num_pages = min_pages;
    a.Hq = num_q_heads;
    a.Hkv = Hkv;
    a.G = pl.G;
    a.max_pages = max_pages_per_seq;
    a.n_clamp = static_cast<int>(std::min<long long>(max_seq_len, 1LL * max_pages_per_seq * kPage));
    a.T = pl.T;
    a.max_splits = pl.max_splits;
    a.out_f32 = out_dtype == PHS_OUT_F32;
    a.scale_log2 = scale_log2;
    // 8 warps per CTA only if all Full layers' grids together fit one wave
    a.num_sms = 1LL * batch * Hkv * pl.max_splits * nfull <= di.sms ? di.sms : 0;
    MergeArgs& ma = m->a;
    ma.seq_lens = seq_lens;
    ma.Hq = num_q_heads;
    ma.Hkv = Hkv;
    ma.G = pl.G;
    ma.n_clamp = a.n_clamp;
    ma.T = pl.T;
    ma.max_splits = pl.max_splits;
    ma.out_f32 = a.out_f32;
    const size_t off_ml = ws_o_bytes(batch, Hkv, pl.max_splits, pl.G, D);
    char* ws = reinterpret_cast<char*>(workspace);
    int k = 0, done = 0;
    st = PHS_OK;
    for (int i = 0; i < num_layers && st == PHS_OK; ++i) {
      const phs_layer& L = layers[i];
      if (!L.is_full) continue;
      StackFullLayer& F = p->layer[k];
      const int64_t rows = L.paged.num_pages * Hkv * kPage;
      if ((st = map_bf16_kv(&F.tk, L.paged.k, rows, D))) break;
      if ((st = map_bf16_kv(&F.tv, L.paged.v, rows, D))) break;
      char* lw = ws + pl.need * static_cast<size_t>(done + k);
      F.q = reinterpret_cast<const __nv_bfloat16*>(L.q);
      F.out = L.out;
      F.ws_o = reinterpret_cast<float*>(lw);
      F.ws_ml = reinterpret_cast<float*>(lw + off_ml);
      F.app = FusedAppend{reinterpret_cast<const __nv_bfloat16*>(L.k_new),
                          reinterpret_cast<const __nv_bfloat16*>(L.v_new),
                          reinterpret_cast<__nv_bfloat16*>(L.paged.k),
                          reinterpret_cast<__nv_bfloat16*>(L.paged.v)};
      m->layer[k] = StackMergeLayer{F.ws_o, F.ws_ml, L.out};
      if (++k == kStackMaxFull) {
        p->num_layers = k;
        if ((st = launch_stack_full(D, *p, batch, s))) break;
        if (pl.max_splits > 1 && (st = launch_stack_merge(D, *m, batch, k, s))) break;
        done += k;
        k = 0;
      }
    }
    if (st == PHS_OK && k) {
      p->num_layers = k;
      if (small)
        small->full = *p;  // launched with the SWA layers below
      else
        st = launch_stack_full(D, *p, batch, s);
      // the last batch of Full layers is merged by the SWA launch when there
      // is one (two launches per step); otherwise by a merge launch
      if (st == PHS_OK && pl.max_splits > 1) {
        if (nswa) {
          fold_merges = *m;
          fold_layers = k;
        } else {
          st = launch_stack_merge(D, *m, batch, k, s);
        }
      }
    }
    delete p;
    delete m;
    if (st) return st;
  }

  // ---- launch 2: every SWA layer (one persistent launch per 64 layers),
  // each unit holding a request's newest slot also appends it
  if (nswa) {
    SwaParams<kSwaMaxLayers>* p = new SwaParams<kSwaMaxLayers>();
    std::memset(p, 0, sizeof(*p));
    p->ring_ids = ring_ids;
    p->ring_pos = ring_pos;
    p->seq_lens = seq_lens;
    p->status = dev_status;
    p->B = batch;
    p->Hq = num_q_heads;
    p->Hkv = Hkv;
    p->G = num_q_heads / Hkv;
    p->W = W;
    p->out_f32 = out_dtype == PHS_OUT_F32;
    p->scale_log2 = scale_log2;
    p->wait_prior_at_exit = nfull > 0;  // every SWA launch here is a dependent launch
    if (fold_layers) {  // the Full layers' merges ride on the first SWA launch
      for (int i = 0; i < fold_layers; ++i) p->merge_layer[i] = fold_merges.layer[i];
      p->merge = fold_merges.a;
      p->num_merge_layers = fold_layers;
    }
    st = PHS_OK;
    for (int i = 0; i < num_layers && st == PHS_OK; ++i) {
      const phs_layer& L = layers[i];
      if (L.is_full) continue;
      const int k = p->num_layers;
      const int64_t rows = L.ring.num_rings * Hkv * W;
      if ((st = map_bf16_kv(&p->tk[k], L.ring.k, rows, D))) break;
      if ((st = map_bf16_kv(&p->tv[k], L.ring.v, rows, D))) break;
      p->q[k] = reinterpret_cast<const __nv_bfloat16*>(L.q);
      p->out[k] = L.out;
      p->num_rings[k] = L.ring.num_rings;
      p->app[k] = FusedAppend{reinterpret_cast<const __nv_bfloat16*>(L.k_new),
                              reinterpret_cast<const __nv_bfloat16*>(L.v_new),
                              reinterpret_cast<__nv_bfloat16*>(L.ring.k),
                              reinterpret_cast<__nv_bfloat16*>(L.ring.v)};
      if (++p->num_layers == kSwaMaxLayers) {
        st = launch_swa_decode<kSwaMaxLayers>(D, *p, di.sms, di.smem_optin, s, nfull > 0);
        p->num_layers = 0;
        p->num_merge_layers = 0;
      }
    }
    if (st == PHS_OK && p->num_layers) {
      if (small) {
        small->swa = *p;
        small->B = batch;
        small->full_ctas = batch * Hkv * nfull;
        st = launch_stack_small(D, *small, batch * Hkv * p->num_layers, s);
      } else {
        st = launch_swa_decode<kSwaMaxLayers>(D, *p, di.sms, di.smem_optin, s, nfull > 0);
      }
    }
    delete p;
    if (st) return st;
  }
  return PHS_OK;
}

int phs_hybrid_kv_tokens(const int32_t* layer_is_full_host, int32_t num_layers,
                         const int32_t* seq_lens_host, int32_t batch, int32_t window,
                         int64_t* full_tokens, int64_t* swa_tokens) {
  if (!layer_is_full_host || !seq_lens_host || !full_tokens || !swa_tokens) return PHS_EINVAL;
  if (num_layers < 0 || batch < 0 || window <= 0) return PHS_EINVAL;
  int64_t f = 0, w = 0;
  for (int l = 0; l < num_layers; ++l)
    for (int b = 0; b < batch; ++b) {
      const int64_t n = seq_lens_host[b] > 0 ? seq_lens_host[b] : 0;
      if (layer_is_full_host[l])
        f += n;
      else
        w += std::min<int64_t>(n, window);
    }
  *full_tokens = f;
  *swa_tokens = w;
  return PHS_OK;
}

int phs_copy_pages(const phs_paged_pool* pool, const int32_t* src_pages, const int32_t* dst_pages,
                   int32_t n, int32_t* dev_status, void* stream) {
  int st = check_paged(pool);
  if (st) return st;
  if (n < 0 || (n > 0 && (!src_pages || !dst_pages))) return PHS_EINVAL;
  const int page_bytes = pool->num_kv_heads * kPage * pool->head_dim * 2;
  return launch_copy_pages(pool->k, pool->v, src_pages, dst_pages, n, pool->num_pages,
                           page_bytes, dev_status, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"

namespace phs {
namespace {

// Shared checks and launch of the SWA segment save / seed calls.
int swa_segment_call(const phs_ring_pool* rings, const phs_paged_pool* segs, int32_t num_layers,
                     SegCopyParams<kSegMaxLayers>& p, int count, cudaStream_t s) {
  if (!rings || !segs || num_layers <= 0) return PHS_EINVAL;
  int st;
  for (int l = 0; l < num_layers; ++l) {
    if ((st = check_ring(&rings[l]))) return st;
    if ((st = check_paged(&segs[l]))) return st;
    if (rings[l].window != rings[0].window || rings[l].num_kv_heads != rings[0].num_kv_heads ||
        rings[l].head_dim != rings[0].head_dim || segs[l].num_kv_heads != rings[0].num_kv_heads ||
        segs[l].head_dim != rings[0].head_dim)
      return PHS_ESHAPE;
  }
  if (count == 0) return PHS_OK;
  p.Hkv = rings[0].num_kv_heads;
  p.D = rings[0].head_dim;
  p.W = rings[0].window;
  for (int l0 = 0; l0 < num_layers; l0 += kSegMaxLayers) {
    p.num_layers = std::min(kSegMaxLayers, num_layers - l0);
    for (int k = 0; k < p.num_layers; ++k) {
      const phs_ring_pool& R = rings[l0 + k];
      const phs_paged_pool& S = segs[l0 + k];
      p.layer[k] = SegCopyLayer{R.k, R.v, S.k, S.v, R.num_rings, S.num_pages};
    }
    if ((st = launch_swa_segment<kSegMaxLayers>(p, count, s))) return st;
  }
  return PHS_OK;
}

}  // namespace
}  // namespace phs

extern "C" {

int phs_swa_ring_save(const phs_ring_pool* rings, const phs_paged_pool* segs, int32_t num_layers,
                      const int32_t* ring_ids, const int32_t* ring_pos, const int32_t* seq_lens,
                      const int32_t* page_index, const int32_t* seg_pages, int32_t count,
                      int32_t* dev_status, void* stream) {
  if (count < 0 || (count > 0 && (!ring_ids || !ring_pos || !seq_lens || !page_index ||
                                   !seg_pages)))
    return PHS_EINVAL;
  SegCopyParams<kSegMaxLayers>* p = new SegCopyParams<kSegMaxLayers>();
  std::memset(p, 0, sizeof(*p));
  p->ring_ids = ring_ids;
  p->ring_pos = ring_pos;
  p->seq_lens = seq_lens;
  p->page_index = page_index;
  p->seg_pages = seg_pages;
  p->status = dev_status;
  p->save = 1;
  const int st = swa_segment_call(rings, segs, num_layers, *p, count,
                                  reinterpret_cast<cudaStream_t>(stream));
  delete p;
  return st;
}

int phs_swa_ring_seed(const phs_ring_pool* rings, const phs_paged_pool* segs, int32_t num_layers,
                      const int32_t* ring_ids, const int32_t* ring_pos, const int32_t* seq_lens,
                      const int32_t* seg_table, int32_t max_seg_pages, int32_t batch,
                      int32_t* dev_status, void* stream) {
  if (batch < 0 || (batch > 0 && (!ring_pos || !seq_lens || !seg_table || max_seg_pages <= 0)))
    return PHS_EINVAL;
  SegCopyParams<kSegMaxLayers>* p = new SegCopyParams<kSegMaxLayers>();
  std::memset(p, 0, sizeof(*p));
  p->ring_ids = ring_ids;
  p->ring_pos = ring_pos;
  p->seq_lens = seq_lens;
  p->seg_table = seg_table;
  p->max_seg = max_seg_pages;
  p->status = dev_status;
  p->save = 0;
  const int st = swa_segment_call(rings, segs, num_layers, *p, batch,
                                  reinterpret_cast<cudaStream_t>(stream));
  delete p;
  return st;
}

int phs_copy_d2d(void* dst, const void* src, size_t bytes, void* stream) {
  if (!dst || !src) return PHS_EINVAL;
  if (!aligned16(dst) || !aligned16(src) || (bytes & 15u)) return PHS_EALIGN;
  DevInfo di;
  int st = dev_info(di);
  if (st) return st;
  return launch_copy(dst, src, bytes, di.sms, reinterpret_cast<cudaStream_t>(stream));
}

int phs_read_checksum(const void* src, size_t bytes, uint32_t* dev_sink, void* stream) {
  if (!src || !dev_sink) return PHS_EINVAL;
  if (!aligned16(src) || (bytes & 15u)) return PHS_EALIGN;
  if ((reinterpret_cast<uintptr_t>(dev_sink) & 3u) != 0) return PHS_EALIGN;
  DevInfo di;
  int st = dev_info(di);
  if (st) return st;
  return launch_read(src, bytes, di.sms, dev_sink, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"

// ---------------------------------------------------------------------------
// No-allocation decode.  The split partials go to this file-scope array
// instead of a caller workspace.  In host code the array's name is only a
// stand-in: its device address is looked up once per device with
// cudaGetSymbolAddress and passed to the kernels.
// ---------------------------------------------------------------------------
static __device__ __align__(256) unsigned char phs_noalloc_scratch[PHS_NOALLOC_SCRATCH_BYTES];

namespace phs {
namespace {

using CtxGetCurrentFn = CUresult (*)(CUcontext*);
using CtxGetIdFn = CUresult (*)(CUcontext, unsigned long long*);

// Unique id of the calling thread's current CUDA context (0 if none or on
// failure).  A context re-created after a device reset gets a new id, so a
// cached device address is never reused across contexts.
unsigned long long current_context_id() {
  static std::once_flag once;
  static CtxGetCurrentFn get_current = nullptr;
  static CtxGetIdFn get_id = nullptr;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      get_current = reinterpret_cast<CtxGetCurrentFn>(p);
    p = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuCtxGetId", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      get_id = reinterpret_cast<CtxGetIdFn>(p);
  });
  if (!get_current || !get_id) return 0;
  CUcontext ctx = nullptr;
  unsigned long long id = 0;
  if (get_current(&ctx) != CUDA_SUCCESS || !ctx) return 0;
  if (get_id(ctx, &id) != CUDA_SUCCESS) return 0;
  return id;
}

// Device address of the scratch in the current context: looked up with
// cudaGetSymbolAddress on the first call in each context (after a device
// reset the new context looks it up again), or null if the lookup fails.
void* noalloc_scratch_on_current_device() {
  static std::mutex mu;
  static std::map<unsigned long long, void*> addr;  // context id -> address
  const unsigned long long id = current_context_id();
  std::lock_guard<std::mutex> lock(mu);
  if (id != 0) {
    auto it = addr.find(id);
    if (it != addr.end()) return it->second;
  }
  // first call in this context (or no context yet: the lookup makes the
  // device's primary context current)
  void* p = nullptr;
  if (cudaGetSymbolAddress(&p, phs_noalloc_scratch) != cudaSuccess) return nullptr;
  const unsigned long long now = current_context_id();
  if (now != 0) addr[now] = p;
  return p;
}

}  // namespace
}  // namespace phs

extern "C" int phs_attn_decode_full_paged_noalloc(
    const void* q, int32_t num_q_heads, const phs_paged_pool* pool, const int32_t* block_table,
    int32_t max_pages_per_seq, const int32_t* seq_lens, int32_t max_seq_len,
    const phs_int8_pool* int8, const int32_t* qtable, int32_t max_qpages_per_seq,
    const int32_t* qlens, int32_t batch, float softmax_scale, int32_t tokens_per_split, void* out,
    int32_t out_dtype, int32_t* dev_status, void* stream) {
  int st = check_paged(pool);
  if (st) return st;
  // choose a split length whose partials fit the scratch
  const bool has_int8 = int8 != nullptr;
  DecodePlan pl;
  if ((st = make_plan(pl, batch, num_q_heads, pool->num_kv_heads, pool->head_dim, max_seq_len,
                      tokens_per_split, has_int8)))
    return st;
  int tps = pl.T;
  while (pl.need > PHS_NOALLOC_SCRATCH_BYTES && tokens_per_split == 0 && tps < kMaxSplitTokens) {
    tps *= 2;
    if ((st = make_plan(pl, batch, num_q_heads, pool->num_kv_heads, pool->head_dim, max_seq_len,
                        tps, has_int8)))
      return st;
  }
  if (pl.need > PHS_NOALLOC_SCRATCH_BYTES) return PHS_ESCRATCH;
  void* scratch = noalloc_scratch_on_current_device();
  if (!scratch) return PHS_ECUDA;
  DecodeCall c;
  st = prepare_decode(c, q, num_q_heads, pool, block_table, max_pages_per_seq, seq_lens,
                      max_seq_len, int8, qtable, max_qpages_per_seq, qlens, batch, softmax_scale,
                      tps, out, out_dtype, scratch, PHS_NOALLOC_SCRATCH_BYTES, nullptr, nullptr,
                      nullptr, dev_status);
  if (st) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if ((st = launch_split_decode(c.pl.D, c.tk, c.tv, c.tk8, c.tv8, c.a, batch, s))) return st;
  if (c.pl.max_splits == 1) return PHS_OK;  // every request finished in its only split
  return launch_merge(c.pl.D, c.m, batch, s);
}

// ------------------------------------------------------ page operations --
namespace {

int check_tables(const void* block_table, const void* seq_lens, int32_t num_rows,
                 int32_t max_pages) {
  if (!block_table || !seq_lens) return PHS_EINVAL;
  if (num_rows <= 0 || max_pages <= 0) return PHS_EINVAL;
  // lengths in tokens are int32
  return max_pages > INT32_MAX / kPage ? PHS_EUNSUPPORTED : PHS_OK;
}

int check_pools(const phs_paged_pool* pools, int32_t num_layers) {
  if (!pools || num_layers <= 0) return PHS_EINVAL;
  for (int32_t l = 0; l < num_layers; ++l) {
    const int st = check_paged(pools + l);
    if (st) return st;
    if (pools[l].num_pages != pools[0].num_pages ||
        pools[l].num_kv_heads != pools[0].num_kv_heads ||
        pools[l].head_dim != pools[0].head_dim)
      return PHS_ESHAPE;
  }
  return PHS_OK;
}

// The pools of a page operation from layer l0 on, as many as a launch takes.
PagePools pools_from(const phs_paged_pool* pools, int32_t num_layers, int32_t l0) {
  PagePools p;
  std::memset(&p, 0, sizeof(p));
  p.num_layers = std::min(num_layers - l0, kPagesMaxLayers);
  p.page_vecs = pools[0].num_kv_heads * kPage * pools[0].head_dim * 2 / 16;
  for (int l = 0; l < p.num_layers; ++l) {
    p.k[l] = reinterpret_cast<uint4*>(pools[l0 + l].k);
    p.v[l] = reinterpret_cast<uint4*>(pools[l0 + l].v);
  }
  return p;
}

// Consecutive 256-byte-aligned int32 arrays of a workspace.
struct Carve {
  char* at;
  size_t used = 0;
  int32_t* take(int64_t n) {
    int32_t* p = reinterpret_cast<int32_t*>(at + used);
    used += align256(static_cast<size_t>(n) * sizeof(int32_t));
    return p;
  }
};

int check_workspace(const void* workspace, size_t bytes, size_t need) {
  if (!workspace || bytes < need) return PHS_EWORKSPACE;
  return (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ? PHS_EALIGN : PHS_OK;
}

}  // namespace

extern "C" {

int phs_pages_free(const int32_t* block_table, int32_t num_rows, int32_t max_pages_per_seq,
                   int32_t* seq_lens, int32_t* page_refcount, int64_t num_pages,
                   const int32_t* rows, int32_t n, int32_t* dev_status, void* stream) {
  const int st = check_tables(block_table, seq_lens, num_rows, max_pages_per_seq);
  if (st) return st;
  if (!page_refcount || num_pages <= 0 || num_pages > INT32_MAX || n < 0 || (n > 0 && !rows))
    return PHS_EINVAL;
  if (n == 0) return PHS_OK;
  const PageFreeArgs a{block_table, seq_lens, page_refcount,     rows, dev_status,
                       num_pages,   num_rows, max_pages_per_seq, n};
  return launch_pages_free(a, reinterpret_cast<cudaStream_t>(stream));
}

size_t phs_pages_fork_workspace_bytes(int32_t num_rows, int32_t n) {
  if (num_rows <= 0 || n < 0) return 0;
  return 2 * align256(static_cast<size_t>(num_rows) * 4) + 4 * align256(static_cast<size_t>(n) * 4);
}

int phs_pages_fork(const phs_paged_pool* pools, int32_t num_layers, int32_t* block_table,
                   int32_t num_rows, int32_t max_pages_per_seq, int32_t* seq_lens,
                   int32_t* page_refcount, const int32_t* src_rows, const int32_t* dst_rows,
                   int32_t n, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                   void* stream) {
  int st = check_pools(pools, num_layers);
  if (st) return st;
  if ((st = check_tables(block_table, seq_lens, num_rows, max_pages_per_seq))) return st;
  if (!page_refcount || n < 0 || (n > 0 && (!src_rows || !dst_rows))) return PHS_EINVAL;
  if (n == 0) return PHS_OK;
  if ((st = check_workspace(workspace, workspace_bytes,
                            phs_pages_fork_workspace_bytes(num_rows, n))))
    return st;
  PageForkArgs a;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.refcount = page_refcount;
  a.src_rows = src_rows;
  a.dst_rows = dst_rows;
  a.status = dev_status;
  a.num_pages = pools[0].num_pages;
  a.num_rows = num_rows;
  a.max_pages = max_pages_per_seq;
  a.n = n;
  Carve ws{reinterpret_cast<char*>(workspace)};
  a.first_dst = ws.take(num_rows);
  a.is_src = ws.take(num_rows);
  a.rank = ws.take(n);
  a.fresh = ws.take(n);
  a.copy_src = ws.take(n);
  a.copy_dst = ws.take(n);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  DevInfo di;
  if ((st = dev_info(di))) return st;
  st = launch_pages_fork(a, pools_from(pools, num_layers, 0), di.sms, s);
  for (int32_t l = kPagesMaxLayers; !st && l < num_layers; l += kPagesMaxLayers)
    st = launch_pages_copy(pools_from(pools, num_layers, l), a.copy_src, a.copy_dst, nullptr, n,
                           di.sms, s);
  return st;
}

size_t phs_pages_compact_workspace_bytes(int64_t num_pages) {
  if (num_pages <= 0 || num_pages > INT32_MAX) return 0;
  return 3 * align256(static_cast<size_t>(num_pages) * 4) + 256 +
         align256(static_cast<size_t>((num_pages + kPagesTile - 1) / kPagesTile) * 4);
}

int phs_pages_compact(const phs_paged_pool* pools, int32_t num_layers,
                      const int32_t* block_table, int32_t num_rows, int32_t max_pages_per_seq,
                      const int32_t* seq_lens, const int32_t* page_refcount,
                      int32_t* block_table_out, int32_t* page_refcount_out, int32_t* page_map,
                      int32_t* num_live, void* workspace, size_t workspace_bytes,
                      int32_t* dev_status, void* stream) {
  int st = check_pools(pools, num_layers);
  if (st) return st;
  if ((st = check_tables(block_table, seq_lens, num_rows, max_pages_per_seq))) return st;
  if (!page_refcount || !block_table_out || !page_refcount_out || !page_map || !num_live)
    return PHS_EINVAL;
  if ((st = check_workspace(workspace, workspace_bytes,
                            phs_pages_compact_workspace_bytes(pools[0].num_pages))))
    return st;
  PageCompactArgs a;
  a.block_table = block_table;
  a.block_table_out = block_table_out;
  a.seq_lens = seq_lens;
  a.refcount = page_refcount;
  a.refcount_out = page_refcount_out;
  a.page_map = page_map;
  a.num_live = num_live;
  a.status = dev_status;
  a.num_pages = pools[0].num_pages;
  a.num_rows = num_rows;
  a.max_pages = max_pages_per_seq;
  Carve ws{reinterpret_cast<char*>(workspace)};
  a.move = ws.take(a.num_pages);
  a.movers = ws.take(a.num_pages);
  a.holes = ws.take(a.num_pages);
  a.meta = ws.take(2);
  a.tile_live = ws.take((a.num_pages + kPagesTile - 1) / kPagesTile);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  DevInfo di;
  if ((st = dev_info(di))) return st;
  st = launch_pages_compact(a, pools_from(pools, num_layers, 0), di.sms, s);
  for (int32_t l = kPagesMaxLayers; !st && l < num_layers; l += kPagesMaxLayers)
    st = launch_pages_copy(pools_from(pools, num_layers, l), a.movers, a.holes, a.meta + 1,
                           a.num_pages / 2, di.sms, s);
  return st;
}

// ------------------------------------------------ differential attention --
}  // extern "C"

namespace {

static_assert(kDiffMaxSplit == kMaxSplitTokens, "the split kernel's chunk lists");

// Split length of a call, with P = batch x value heads (x 2 for groups of more
// than 8 heads) and a wave of W = SMs x CTAs of an SM.
// Where one wave can hold every split, the length that just does (in whole
// steps of 128): the call then has one round of CTAs and few partials.  (us:
// one request of 250,001 tokens, 4 value heads of 64: 147 at 256 tokens a
// split, 100 at 1,024, 108.9 at 2,048, which is 1.08 waves, 87 at 2,208, 84 at
// 4,096; 4 requests of 32K on one of 128: 39.2 at 512, 29.5 at 896, 47.1 at
// 2,048; one of 8K on 4 of 128: 18.9 at 128, 12.6 at 256, 15.9 at 512.)
// Else, and where a batch may be so ragged that one wave would leave most of
// it empty (the length above is over four times the one below), the length T
// that balances what a CTA costs beside its bytes, about 3 us, N / (T W)
// times in a row for N tokens in all, against half a CTA at the end, T / 2
// tokens of 8 D bytes on all W at 7.1 TB/s.  N is taken as half of what the
// stated bound allows.  (64 requests to 32K: 378 at 1,024, 367 at 2,048, 372
// at 4,096; 16 to 4K: 21.4 at 256, 20.2 at 512, 68 at 4,096, the one wave.)
int plan_diff_split(int B, int Hv, int G, int D, int max_seq, int sms) {
  const double pairs = 1.0 * B * Hv * ((G + 7) / 8), wave = 1.0 * sms * diff_ctas_per_sm(D);
  const double tokens = pairs * max_seq / (B == 1 ? 1 : 2);
  const double best = std::sqrt(3.0 * tokens * 7.1e6 / (4.0 * D * wave * wave));
  const int per = static_cast<int>(wave / pairs);  // splits of a request in one wave
  if (per > 0) {
    const int one = std::max(1, ((max_seq + per - 1) / per + 127) / 128) * 128;
    if (one <= kDiffMaxSplit && (B == 1 || one <= 4 * best)) return one;
  }
  int T = 128;
  while (T < kDiffMaxSplit && T * 1.5 < best) T *= 2;  // the nearest power of two
  return T;
}

int make_diff_plan(DecodePlan& pl, int B, int H, int Hv, int D, int max_seq, int tps) {
  int st = make_plan(pl, B, H, Hv, D, max_seq, tps, false);
  if (st || tps > 0) return st;
  DevInfo di;
  if ((st = dev_info(di))) return st;
  return make_plan(pl, B, H, Hv, D, max_seq, plan_diff_split(B, Hv, pl.G, D, max_seq, di.sms),
                   false);
}

// Partials of a split: one 2D-wide row and one (max, sum) for each map of
// each head.  A call that needs none (one split) still takes a workspace.
size_t diff_rows(const DecodePlan& pl, int B) {
  return static_cast<size_t>(B) * pl.Hkv * pl.max_splits * pl.G * 2;
}
size_t diff_o_bytes(const DecodePlan& pl, int B) {
  return align256(diff_rows(pl, B) * 2 * pl.D * sizeof(float));
}

}  // namespace

extern "C" {

size_t phs_diff_workspace_bytes(int32_t batch, int32_t num_heads, int32_t num_value_heads,
                                int32_t head_dim, int32_t max_seq_len,
                                int32_t tokens_per_split) {
  DecodePlan pl;
  if (make_diff_plan(pl, batch, num_heads, num_value_heads, head_dim, max_seq_len,
                     tokens_per_split))
    return 0;
  return diff_o_bytes(pl, batch) + align256(diff_rows(pl, batch) * 2 * sizeof(float));
}

int phs_attn_decode_diff_paged(const void* q, int32_t num_heads, const phs_paged_pool* pool,
                               const int32_t* block_table, int32_t max_pages_per_seq,
                               const int32_t* seq_lens, int32_t max_seq_len, int32_t batch,
                               const phs_diff_weights* weights, float softmax_scale,
                               int32_t tokens_per_split, void* out, int32_t out_dtype,
                               void* workspace, size_t workspace_bytes, const void* k_new,
                               const void* v_new, const int32_t* page_refcount,
                               int32_t* dev_status, void* stream) {
  int st = check_paged(pool);
  if (st) return st;
  if (!q || !block_table || !seq_lens || !out || !weights) return PHS_EINVAL;
  if (!weights->lambda_q1 || !weights->lambda_k1 || !weights->lambda_q2 || !weights->lambda_k2)
    return PHS_EINVAL;
  if (!std::isfinite(weights->lambda_init) || !(weights->norm_eps >= 0.f) ||
      !std::isfinite(weights->norm_eps))
    return PHS_EINVAL;
  if ((k_new == nullptr) != (v_new == nullptr)) return PHS_EINVAL;
  if (k_new && (!aligned16(k_new) || !aligned16(v_new))) return PHS_EALIGN;
  if (max_pages_per_seq <= 0 || !(softmax_scale > 0.f) || !std::isfinite(softmax_scale))
    return PHS_EINVAL;
  if (out_dtype != PHS_OUT_BF16 && out_dtype != PHS_OUT_F32) return PHS_EINVAL;
  if (pool->num_kv_heads % 2 != 0) return PHS_ESHAPE;
  const int Hv = pool->num_kv_heads / 2, D = pool->head_dim;
  DecodePlan pl;
  if ((st = make_diff_plan(pl, batch, num_heads, Hv, D, max_seq_len, tokens_per_split)))
    return st;
  if ((st = check_workspace(workspace, workspace_bytes,
                            phs_diff_workspace_bytes(batch, num_heads, Hv, D, max_seq_len,
                                                     tokens_per_split))))
    return st;
  if (!aligned16(q) || !aligned16(out)) return PHS_EALIGN;
  DiffArgs a;
  std::memset(&a, 0, sizeof(a));
  a.q = reinterpret_cast<const __nv_bfloat16*>(q);
  a.k = reinterpret_cast<__nv_bfloat16*>(pool->k);
  a.v = reinterpret_cast<__nv_bfloat16*>(pool->v);
  a.k_new = reinterpret_cast<const __nv_bfloat16*>(k_new);
  a.v_new = reinterpret_cast<const __nv_bfloat16*>(v_new);
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.page_refcount = page_refcount;
  a.out = out;
  a.ws_o = reinterpret_cast<float*>(workspace);
  a.ws_ml = reinterpret_cast<float*>(reinterpret_cast<char*>(workspace) + diff_o_bytes(pl, batch));
  a.T = pl.T;
  a.max_splits = pl.max_splits;
  a.status = dev_status;
  a.num_pages = pool->num_pages;
  a.H = num_heads;
  a.Hv = Hv;
  a.G = num_heads / Hv;
  a.max_pages = max_pages_per_seq;
  a.n_clamp = static_cast<int>(std::min<long long>(max_seq_len, 1LL * max_pages_per_seq * kPage));
  a.out_f32 = out_dtype == PHS_OUT_F32;
  a.scale_log2 = softmax_scale * 1.4426950408889634f;
  a.lambda_q1 = weights->lambda_q1;
  a.lambda_k1 = weights->lambda_k1;
  a.lambda_q2 = weights->lambda_q2;
  a.lambda_k2 = weights->lambda_k2;
  a.norm_weight = weights->norm_weight;
  a.lambda_init = weights->lambda_init;
  a.norm_eps = weights->norm_eps;
  a.lambda_per_head = weights->lambda_per_head != 0;
  CUtensorMap tk, tv;
  const int64_t rows = pool->num_pages * pool->num_kv_heads * kPage;
  if ((st = map_bf16_kv(&tk, pool->k, rows, D, 2 * kPage))) return st;
  if ((st = map_bf16_kv(&tv, pool->v, rows, D, 2 * kPage))) return st;
  return launch_diff_decode(D, tk, tv, a, batch, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"

// ------------------------------------------------------ linear attention --
namespace {

int linear_args(LinearArgs& a, const void* q, int32_t num_q_heads, const void* k, const void* v,
                const phs_state_pool* pool, const int32_t* state_ids, const float* log_decay,
                int32_t batch, int32_t tokens, float scale, void* out, int32_t out_dtype,
                int32_t* dev_status) {
  if (!pool || !pool->s || pool->num_states <= 0 || pool->num_kv_heads <= 0) return PHS_EINVAL;
  if (!log_decay || batch < 0 || tokens < 0 || !std::isfinite(scale)) return PHS_EINVAL;
  if (tokens > 0 && (!q || !k || !v || !out)) return PHS_EINVAL;
  if (out_dtype != PHS_OUT_BF16 && out_dtype != PHS_OUT_F32) return PHS_EINVAL;
  const int st = check_dims(num_q_heads, pool->num_kv_heads, pool->head_dim);
  if (st) return st;
  if (pool->num_kv_heads > 65535) return PHS_EUNSUPPORTED;  // grid y
  if (!state_ids && batch > pool->num_states) return PHS_ESHAPE;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned16(pool->s))
    return PHS_EALIGN;
  std::memset(&a, 0, sizeof(a));
  a.q = reinterpret_cast<const __nv_bfloat16*>(q);
  a.k = reinterpret_cast<const __nv_bfloat16*>(k);
  a.v = reinterpret_cast<const __nv_bfloat16*>(v);
  a.state = pool->s;
  a.log_decay = log_decay;
  a.state_ids = state_ids;
  a.out = out;
  a.status = dev_status;
  a.num_states = pool->num_states;
  a.Hq = num_q_heads;
  a.Hkv = pool->num_kv_heads;
  a.G = num_q_heads / pool->num_kv_heads;
  a.B = batch;
  a.out_f32 = out_dtype == PHS_OUT_F32;
  a.scale = scale;
  return PHS_OK;
}

}  // namespace

extern "C" {

int phs_linear_attn_decode(const void* q, int32_t num_q_heads, const phs_state_pool* pool,
                           const void* k_new, const void* v_new, const float* log_decay,
                           const int32_t* state_ids, int32_t batch, float scale, void* out,
                           int32_t out_dtype, int32_t* dev_status, void* stream) {
  LinearArgs a;
  const int st = linear_args(a, q, num_q_heads, k_new, v_new, pool, state_ids, log_decay, batch,
                             batch, scale, out, out_dtype, dev_status);
  if (st || batch == 0) return st;
  return launch_linear_decode(pool->head_dim, a, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"

namespace {

// The cheaper of no segments of each prompt and as many as leave each CTA an SM to
// itself, with the parts that a first launch sums a segment up in (shared by the
// chunked prompt calls).  A call has `pairs` (request, unit of heads), `groups` CTAs
// for each; the longest request has `chunks`, all units of all requests
// `all_chunks`.  Costs in half microseconds: 16 for a CTA (of either launch); for a
// chunk `chunk`, of which 4 for its state (in either launch); 4 for joining the sums.
struct Segments {
  long long time = -1;
  int nseg = 1, nsub = 1;
};
Segments best_segments(long long pairs, int groups, long long chunks, long long all_chunks,
                       long long chunk, int sms) {
  Segments best;
  const long long most = std::max(1LL, std::min(sms / (pairs * groups), chunks / 2));
  for (const long long s : {1LL, most}) {
    const long long per = (chunks + s - 1) / s;
    long long time = 16 + per * chunk, sub = 1;
    if (s == 1) {  // (a request's last chunk is half full on average)
      time = std::max(time, groups * (pairs * 16 + chunk * all_chunks) / sms);
    } else {
      long long sums = -1;
      for (long long n = 1; n <= 8 && n <= per; ++n) {
        const long long waves = ((s - 1) * pairs * n + sms - 1) / sms;
        const long long t = waves * (16 + 4 * ((per + n - 1) / n));
        if (sums >= 0 && t >= sums) continue;
        sums = t;
        sub = n;
      }
      time += sums + 4;
    }
    if (best.time >= 0 && time >= best.time) continue;
    best.time = time;
    best.nseg = static_cast<int>(s);
    best.nsub = static_cast<int>(sub);
  }
  return best;
}

// How a prompt call is spread over the SMs: segments of each prompt, parts
// that a first launch sums a segment up in, and CTAs that share a KV head's
// query heads.  Of the plans the one with the least time is taken, by these
// costs at D = 128 (taken at 64 too) in half microseconds: 16 for a CTA (of either launch); for
// each chunk 4 for its state (in either launch) and 3 for each query head of
// the CTA; 4 for joining the sums.  Without segments a call takes as long as
// its longest prompt, or as all CTAs' work spread over the SMs; segments are
// only made while each CTA has an SM to itself.  (One prompt of 32,768 tokens, 8
// heads on one: 76 us, against 139 with segments of 8 chunks each; one of
// 2,048, 8 heads: 28 against 60.)
struct LinearPlan {
  int nseg = 1, nsub = 1, ngrp = 1;
  size_t need = 256;
};
LinearPlan linear_plan(int B, int G, int Hkv, int D, int total, int max_seq, int sms) {
  LinearPlan p;
  const long long pairs = std::max(1LL, 1LL * B * Hkv), C = kLinearChunk;
  const long long chunks = (std::min(total, max_seq) + C - 1) / C;
  long long best = -1;
  for (int g = 1; g <= G; ++g) {
    if (G % g != 0) continue;
    const Segments s =
        best_segments(pairs, g, chunks, Hkv * (total / C + B / 2), 4 + 3 * (G / g), sms);
    if (best >= 0 && s.time >= best) continue;
    best = s.time;
    p.nseg = s.nseg;
    p.nsub = s.nsub;
    p.ngrp = g;
  }
  if (p.nseg > 1 || p.ngrp > 1)
    p.need = static_cast<size_t>(pairs) * p.nseg * p.nsub * D * D * sizeof(float);
  return p;
}

// [tokens][heads * D] bf16; boxes of 128 tokens x 64 columns
int map_bf16_tokens(CUtensorMap* m, const void* base, int64_t tokens, int64_t cols) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return PHS_ECUDA;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(tokens)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols) * 2};
  cuuint32_t box[2] = {64, kLinearChunk};
  cuuint32_t es[2] = {1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides,
                   box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? PHS_OK : PHS_ECUDA;
}

}  // namespace

extern "C" {

size_t phs_linear_prompt_workspace_bytes(int32_t batch, int32_t num_q_heads,
                                         int32_t num_kv_heads, int32_t head_dim,
                                         int32_t total_tokens, int32_t max_seq_len) {
  if (batch < 0 || total_tokens < 0 || max_seq_len < 0 ||
      check_dims(num_q_heads, num_kv_heads, head_dim))
    return 0;
  DevInfo di;
  if (dev_info(di)) return 0;
  return linear_plan(batch, num_q_heads / num_kv_heads, num_kv_heads, head_dim, total_tokens,
                     max_seq_len, di.sms)
      .need;
}

int phs_linear_attn_prompt(const void* q, int32_t num_q_heads, const void* k, const void* v,
                           const int32_t* cu_seqlens, int32_t total_tokens, int32_t max_seq_len,
                           const phs_state_pool* pool, const int32_t* state_ids,
                           const int32_t* resume, const float* log_decay, int32_t batch,
                           float scale, void* out, void* workspace, size_t workspace_bytes,
                           int32_t* dev_status, void* stream) {
  LinearArgs a;
  int st = linear_args(a, q, num_q_heads, k, v, pool, state_ids, log_decay, batch,
                       total_tokens, scale, out, PHS_OUT_BF16, dev_status);
  if (st) return st;
  if (!cu_seqlens || max_seq_len < 0) return PHS_EINVAL;
  if (batch == 0) return PHS_OK;
  if ((st = check_workspace(workspace, workspace_bytes,
                            phs_linear_prompt_workspace_bytes(batch, num_q_heads,
                                                              pool->num_kv_heads, pool->head_dim,
                                                              total_tokens, max_seq_len))))
    return st;
  a.cu_seqlens = cu_seqlens;
  a.resume = resume;
  a.total_tokens = total_tokens;
  a.max_seq = max_seq_len;
  DevInfo di;
  if ((st = dev_info(di))) return st;
  const LinearPlan plan =
      linear_plan(batch, a.G, a.Hkv, pool->head_dim, total_tokens, max_seq_len, di.sms);
  a.nseg = plan.nseg;
  a.nsub = plan.nsub;
  a.ngrp = plan.ngrp;
  const int64_t ctas = int64_t{batch} * a.Hkv * a.nseg * a.ngrp;
  if (ctas > INT32_MAX) return PHS_EUNSUPPORTED;
  a.longest_first = ctas > di.sms && batch > 1 && batch <= kLinearSort;
  a.ws = reinterpret_cast<float*>(workspace);
  CUtensorMap tq, tk, tv, to;
  std::memset(&tq, 0, sizeof(tq));
  if (total_tokens > 0) {
    const int D = pool->head_dim;
    if ((st = map_bf16_tokens(&tq, q, total_tokens, int64_t{a.Hq} * D))) return st;
    if ((st = map_bf16_tokens(&tk, k, total_tokens, int64_t{a.Hkv} * D))) return st;
    if ((st = map_bf16_tokens(&tv, v, total_tokens, int64_t{a.Hkv} * D))) return st;
    if ((st = map_bf16_tokens(&to, out, total_tokens, int64_t{a.Hq} * D))) return st;
  } else {
    tk = tv = to = tq;  // no chunk, no copy
  }
  return launch_linear_prompt(pool->head_dim, tq, tk, tv, to, a,
                              reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"

// ----------------------------------------- rotary positions, cache writes --
namespace {

// Rows of `cols` elements at a stride: 16-byte pieces.
bool bad_rows(int64_t stride, int64_t cols) { return stride < cols || stride % 8 != 0; }

// A kernel's last tile ends behind the last row, and a row's elements are
// counted in 32 bits.
bool too_many(int64_t rows, int64_t cols) { return rows > INT32_MAX - 65536 || cols > INT32_MAX; }

// Whether rows of `cols` elements at a stride and others share memory: parts of
// the same wider rows do not; else rows whose ranges meet are taken to.
struct Rows {
  const void* at;
  int64_t stride, cols, size;  // in elements of `size` bytes
};
bool overlap(const Rows& a, const Rows& b, int64_t tokens) {
  if (tokens <= 0 || !a.at || !b.at) return false;
  const uint64_t as = a.stride * a.size, bs = b.stride * b.size;  // bytes
  const uint64_t ac = a.cols * a.size, bc = b.cols * b.size;
  const uint64_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
  if (x + (tokens - 1) * as + ac <= y || y + (tokens - 1) * bs + bc <= x) return false;
  if (as != bs) return true;
  const uint64_t d = y >= x ? (y - x) % as : (as - (x - y) % as) % as;  // b's first column in a's row
  return d < ac || d + bc > as;
}
// The same, where an output may also be its own input.
bool overlap_in_part(const Rows& in, const Rows& out, int64_t tokens) {
  return !(in.at == out.at && (in.stride == out.stride || tokens <= 1)) &&
         overlap(in, out, tokens);
}

int check_rope(const phs_rope* rope, int D) {
  if (!rope->turns || rope->rotary_dim <= 0 || !std::isfinite(rope->factor)) return PHS_EINVAL;
  if (rope->rotary_dim > D) return PHS_ESHAPE;
  if (rope->rotary_dim % 16 != 0) return PHS_EUNSUPPORTED;
  return PHS_OK;
}

void set_rope(WriteArgs& a, const phs_rope* rope) {
  a.turns = rope->turns;
  a.rotary = rope->rotary_dim;
  a.interleaved = rope->interleaved != 0;
  a.factor = rope->factor;
}

int run_write(int D, const WriteArgs& a, void* stream) {
  DevInfo di;
  const int st = dev_info(di);
  return st ? st : launch_write(D, a, di.sms, reinterpret_cast<cudaStream_t>(stream));
}

}  // namespace

extern "C" {

int phs_rope_rotate(const void* q, int64_t q_stride, int32_t num_q_heads, const void* k,
                    int64_t k_stride, int32_t num_kv_heads, int32_t head_dim, int32_t tokens,
                    const int32_t* positions, const phs_rope* rope, void* q_out,
                    int64_t q_out_stride, void* k_out, int64_t k_out_stride, void* stream) {
  if (tokens < 0 || !rope || num_q_heads <= 0 || (k && num_kv_heads <= 0)) return PHS_EINVAL;
  if ((k == nullptr) != (k_out == nullptr)) return PHS_EINVAL;
  if (tokens > 0 && (!q || !q_out || !positions)) return PHS_EINVAL;
  if (head_dim != 64 && head_dim != 128) return PHS_EUNSUPPORTED;
  const int st = check_rope(rope, head_dim);
  if (st) return st;
  const int64_t qc = int64_t{num_q_heads} * head_dim, kc = int64_t{num_kv_heads} * head_dim;
  if (bad_rows(q_stride, qc) || bad_rows(q_out_stride, qc)) return PHS_ESHAPE;
  if (k && (bad_rows(k_stride, kc) || bad_rows(k_out_stride, kc))) return PHS_ESHAPE;
  if (!aligned16(q) || !aligned16(q_out) || !aligned16(k) || !aligned16(k_out)) return PHS_EALIGN;
  if (too_many(tokens, qc) || (k && too_many(tokens, kc))) return PHS_EUNSUPPORTED;
  if (tokens == 0) return PHS_OK;
  const Rows qi{q, q_stride, qc, 2}, ki{k, k_stride, kc, 2};
  const Rows qo{q_out, q_out_stride, qc, 2}, ko{k_out, k_out_stride, kc, 2};
  if (overlap_in_part(qi, qo, tokens) || overlap_in_part(ki, ko, tokens) ||
      overlap(qi, ko, tokens) || overlap(ki, qo, tokens) || overlap(qo, ko, tokens))
    return PHS_EINVAL;
  WriteArgs a;
  std::memset(&a, 0, sizeof(a));
  a.q = reinterpret_cast<const __nv_bfloat16*>(q);
  a.k = reinterpret_cast<const __nv_bfloat16*>(k);
  a.q_out = reinterpret_cast<__nv_bfloat16*>(q_out);
  a.k_out = reinterpret_cast<__nv_bfloat16*>(k_out);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.q_out_stride = q_out_stride;
  a.k_out_stride = k_out_stride;
  a.positions = positions;
  a.Hq = num_q_heads;
  a.Hkv = num_kv_heads;
  a.tokens = tokens;
  set_rope(a, rope);
  return run_write(head_dim, a, stream);
}

int phs_kv_write_paged(const phs_paged_pool* pool, const void* k, int64_t k_stride, const void* v,
                       int64_t v_stride, int32_t tokens, const int32_t* cu_seqlens,
                       const int32_t* block_table, int32_t max_pages_per_seq,
                       const int32_t* seq_lens, int32_t batch, const phs_rope* rope,
                       const void* q, int64_t q_stride, int32_t num_q_heads, void* q_out,
                       const phs_int8_pool* int8, const int32_t* qtable,
                       int32_t max_qpages_per_seq, const int32_t* qlens_before,
                       const int32_t* qlens, int32_t max_qblocks, const int32_t* page_refcount,
                       int32_t* dev_status, void* stream) {
  int st = check_paged(pool);
  if (st) return st;
  if (tokens < 0 || batch < 0 || max_pages_per_seq <= 0) return PHS_EINVAL;
  if (tokens > 0 && (!k || !v)) return PHS_EINVAL;
  if (batch > 0 && (!block_table || !seq_lens)) return PHS_EINVAL;
  if (!cu_seqlens && tokens != batch) return PHS_ESHAPE;
  const int D = pool->head_dim;
  const int64_t kc = int64_t{pool->num_kv_heads} * D;
  if (tokens > 0 && (bad_rows(k_stride, kc) || bad_rows(v_stride, kc))) return PHS_ESHAPE;
  if (!aligned16(k) || !aligned16(v)) return PHS_EALIGN;
  if (too_many(tokens, q ? int64_t{num_q_heads} * D : 0)) return PHS_EUNSUPPORTED;
  if (rope && (st = check_rope(rope, D))) return st;
  if (q) {
    if (!rope || !q_out || num_q_heads <= 0) return PHS_EINVAL;
    if (bad_rows(q_stride, int64_t{num_q_heads} * D)) return PHS_ESHAPE;
    if (!aligned16(q) || !aligned16(q_out)) return PHS_EALIGN;
  }
  WriteArgs a;
  std::memset(&a, 0, sizeof(a));
  if (int8) {
    if ((st = check_int8(int8))) return st;
    if (int8->num_kv_heads != pool->num_kv_heads || int8->head_dim != D) return PHS_ESHAPE;
    if (batch > 0 && (!qtable || !qlens_before || !qlens)) return PHS_EINVAL;
    if (max_qpages_per_seq <= 0 || max_qblocks < 0) return PHS_EINVAL;
    if (batch > 65535 || max_qblocks > INT32_MAX / 64) return PHS_EUNSUPPORTED;  // the grid
    a.k_codes = int8->k;
    a.v_codes = int8->v;
    a.k_scale = int8->k_scale;
    a.v_scale = int8->v_scale;
    a.qtable = qtable;
    a.qlens_before = qlens_before;
    a.qlens = qlens;
    a.num_qpages = int8->num_qpages;
    a.max_qpages = max_qpages_per_seq;
    a.max_qblocks = max_qblocks;
  }
  if (batch == 0) return PHS_OK;
  if (q) {
    const int64_t qc = int64_t{num_q_heads} * D;
    const Rows qo{q_out, qc, qc, 2};
    if (overlap_in_part({q, q_stride, qc, 2}, qo, tokens) ||
        overlap({k, k_stride, kc, 2}, qo, tokens) || overlap({v, v_stride, kc, 2}, qo, tokens))
      return PHS_EINVAL;
  }
  a.q = reinterpret_cast<const __nv_bfloat16*>(q);
  a.k = reinterpret_cast<const __nv_bfloat16*>(k);
  a.v = reinterpret_cast<const __nv_bfloat16*>(v);
  a.q_out = reinterpret_cast<__nv_bfloat16*>(q_out);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_out_stride = int64_t{num_q_heads} * D;
  a.cu_seqlens = cu_seqlens;
  a.seq_lens = seq_lens;
  a.block_table = block_table;
  a.page_refcount = page_refcount;
  a.status = dev_status;
  a.pool_k = reinterpret_cast<__nv_bfloat16*>(pool->k);
  a.pool_v = reinterpret_cast<__nv_bfloat16*>(pool->v);
  a.num_pages = pool->num_pages;
  a.Hq = q ? num_q_heads : 0;
  a.Hkv = pool->num_kv_heads;
  a.tokens = tokens;
  a.B = batch;
  a.max_pages = max_pages_per_seq;
  if (rope) set_rope(a, rope);
  return run_write(D, a, stream);
}

int phs_kv_read_paged(const phs_paged_pool* pool, const int32_t* block_table,
                      int32_t max_pages_per_seq, const int32_t* starts,
                      const int32_t* cu_seqlens, int32_t batch, int32_t tokens,
                      int32_t max_tokens, const phs_int8_pool* int8, const int32_t* qtable,
                      int32_t max_qpages_per_seq, const int32_t* qlens, void* k_out, void* v_out,
                      int32_t* dev_status, void* stream) {
  int st = check_paged(pool);
  if (st) return st;
  if (batch < 0 || tokens < 0 || max_tokens < 0 || max_pages_per_seq <= 0) return PHS_EINVAL;
  if (batch > 0 && (!block_table || !starts || !cu_seqlens)) return PHS_EINVAL;
  if (tokens > 0 && (!k_out || !v_out)) return PHS_EINVAL;
  if (!aligned16(k_out) || !aligned16(v_out)) return PHS_EALIGN;
  if (batch > 65535 || too_many(tokens, 0)) return PHS_EUNSUPPORTED;  // (grid y)
  ReadArgs a;
  std::memset(&a, 0, sizeof(a));
  if (int8) {
    if ((st = check_int8(int8))) return st;
    if (int8->num_kv_heads != pool->num_kv_heads || int8->head_dim != pool->head_dim)
      return PHS_ESHAPE;
    if (max_qpages_per_seq <= 0 || (batch > 0 && (!qtable || !qlens))) return PHS_EINVAL;
    a.k_codes = int8->k;
    a.v_codes = int8->v;
    a.k_scale = int8->k_scale;
    a.v_scale = int8->v_scale;
    a.qtable = qtable;
    a.qlens = qlens;
    a.num_qpages = int8->num_qpages;
    a.max_qpages = max_qpages_per_seq;
  }
  if (batch == 0) return PHS_OK;
  a.pool_k = reinterpret_cast<const __nv_bfloat16*>(pool->k);
  a.pool_v = reinterpret_cast<const __nv_bfloat16*>(pool->v);
  a.block_table = block_table;
  a.starts = starts;
  a.cu_seqlens = cu_seqlens;
  a.status = dev_status;
  a.k_out = reinterpret_cast<__nv_bfloat16*>(k_out);
  a.v_out = reinterpret_cast<__nv_bfloat16*>(v_out);
  a.num_pages = pool->num_pages;
  a.Hkv = pool->num_kv_heads;
  a.B = batch;
  a.tokens = tokens;
  // (no request has more tokens than there are)
  a.max_tokens = std::min(max_tokens, tokens);
  a.max_pages = max_pages_per_seq;
  return launch_read_back(pool->head_dim, a, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"

// ---------------------------------------- causal convolution, selective scan --
namespace {

int conv_args(ConvArgs& a, const void* x, int64_t x_stride, const phs_conv_pool* pool,
              const phs_conv_weights* weights, const int32_t* state_ids, int32_t batch,
              int32_t tokens, void* out, int32_t* dev_status) {
  if (!pool || !pool->c || pool->num_states <= 0 || pool->channels <= 0) return PHS_EINVAL;
  if (!weights || !weights->weight || batch < 0 || tokens < 0) return PHS_EINVAL;
  if (tokens > 0 && (!x || !out)) return PHS_EINVAL;
  if (pool->width < 2 || pool->width > 4 || pool->channels % 8 != 0) return PHS_EUNSUPPORTED;
  if (too_many(tokens, 0)) return PHS_EUNSUPPORTED;
  if (tokens > 0 && bad_rows(x_stride, pool->channels)) return PHS_ESHAPE;
  if (!state_ids && batch > pool->num_states) return PHS_ESHAPE;
  if (!aligned16(x) || !aligned16(out) || !aligned16(pool->c) || !aligned16(weights->weight) ||
      !aligned16(weights->bias))
    return PHS_EALIGN;
  std::memset(&a, 0, sizeof(a));
  a.x = reinterpret_cast<const __nv_bfloat16*>(x);
  a.x_stride = x_stride;
  a.state = reinterpret_cast<__nv_bfloat16*>(pool->c);
  a.weight = weights->weight;
  a.bias = weights->bias;
  a.silu = weights->silu != 0;
  a.state_ids = state_ids;
  a.out = reinterpret_cast<__nv_bfloat16*>(out);
  a.status = dev_status;
  a.num_states = pool->num_states;
  a.channels = pool->channels;
  a.B = batch;
  a.tokens = tokens;
  return PHS_OK;
}

int scan_args(ScanArgs& a, const phs_scan_inputs* in, const phs_scan_pool* pool,
              const phs_scan_weights* weights, const int32_t* state_ids, int32_t batch,
              int32_t tokens, void* out, int32_t out_dtype, int32_t* dev_status) {
  if (!in || !pool || !pool->s || pool->num_states <= 0 || pool->num_heads <= 0) return PHS_EINVAL;
  if (!weights || !weights->a || batch < 0 || tokens < 0 || in->num_groups <= 0) return PHS_EINVAL;
  if (tokens > 0 && (!in->x || !in->b || !in->c || !in->dt || !out)) return PHS_EINVAL;
  if (out_dtype != PHS_OUT_BF16 && out_dtype != PHS_OUT_F32) return PHS_EINVAL;
  if (in->dt_dtype != PHS_OUT_BF16 && in->dt_dtype != PHS_OUT_F32) return PHS_EINVAL;
  const int H = pool->num_heads, G = in->num_groups, P = pool->head_dim, N = pool->state_dim;
  if (H % G != 0) return PHS_ESHAPE;
  if ((P != 64 && P != 128) || (N != 64 && N != 128)) return PHS_EUNSUPPORTED;
  if (H > 65535) return PHS_EUNSUPPORTED;  // grid y
  if (tokens > 0 && (bad_rows(in->x_stride, int64_t{H} * P) ||
                     bad_rows(in->b_stride, int64_t{G} * N) ||
                     bad_rows(in->c_stride, int64_t{G} * N) || in->dt_stride < H))
    return PHS_ESHAPE;
  if (!state_ids && batch > pool->num_states) return PHS_ESHAPE;
  if (!aligned16(in->x) || !aligned16(in->b) || !aligned16(in->c) || !aligned16(out) ||
      !aligned16(pool->s))
    return PHS_EALIGN;
  std::memset(&a, 0, sizeof(a));
  a.x = reinterpret_cast<const __nv_bfloat16*>(in->x);
  a.b = reinterpret_cast<const __nv_bfloat16*>(in->b);
  a.c = reinterpret_cast<const __nv_bfloat16*>(in->c);
  a.dt = in->dt;
  a.x_stride = in->x_stride;
  a.b_stride = in->b_stride;
  a.c_stride = in->c_stride;
  a.dt_stride = in->dt_stride;
  a.dt_f32 = in->dt_dtype == PHS_OUT_F32;
  a.state = pool->s;
  a.rate = weights->a;
  a.skip = weights->skip;
  a.dt_bias = weights->dt_bias;
  a.state_ids = state_ids;
  a.out = out;
  a.status = dev_status;
  a.num_states = pool->num_states;
  a.H = H;
  a.G = G;
  a.B = batch;
  a.out_f32 = out_dtype == PHS_OUT_F32;
  return PHS_OK;
}

bool scan_overlap(const ScanArgs& a, int P, int N, int64_t tokens) {
  const int64_t hp = int64_t{a.H} * P, gn = int64_t{a.G} * N;
  const Rows out{a.out, hp, hp, a.out_f32 ? 4 : 2};
  return overlap({a.x, a.x_stride, hp, 2}, out, tokens) ||
         overlap({a.b, a.b_stride, gn, 2}, out, tokens) ||
         overlap({a.c, a.c_stride, gn, 2}, out, tokens) ||
         overlap({a.dt, a.dt_stride, a.H, a.dt_f32 ? 4 : 2}, out, tokens);
}

// How a prompt call is spread over the SMs: 64-wide heads in pairs where a
// group has an even number of them, and segments by best_segments with 4 half
// microseconds of a chunk for the rows of each slot.
struct ScanPlan {
  int slots = 1, units = 1, nseg = 1, nsub = 1;
  size_t tables = 0, sums = 0, need = 0;  // bytes
};
ScanPlan scan_plan(int B, int H, int G, int P, int N, int total, int max_seq, int sms) {
  ScanPlan p;
  p.slots = P == 128 || H / G % 2 == 0 ? 2 : 1;
  p.units = H * (P / 64) / p.slots;
  const long long pairs = std::max(1LL, 1LL * B * p.units), C = kScanChunk;
  const Segments s = best_segments(pairs, 1, (std::min(total, max_seq) + C - 1) / C,
                                   p.units * (total / C + B / 2), 4 + 4 * p.slots, sms);
  p.nseg = s.nseg;
  p.nsub = s.nsub;
  // (in 64 bits: 65,535 requests of 128 heads have 4.5e9 floats of tables)
  p.tables = align256(static_cast<size_t>(total / C + B + 1) * H * kScanTable * sizeof(float));
  if (p.nseg > 1)
    p.sums = align256(static_cast<size_t>(pairs) * p.nseg * p.nsub * 64 * p.slots * N * sizeof(float));
  p.need = p.tables + p.sums;
  if (p.nseg > 1) p.need += align256(static_cast<size_t>(pairs) * p.nseg * p.nsub * 2 * sizeof(float));
  return p;
}

// Whether every request of a call goes token by token, by one launch that keeps
// nothing in the workspace.
bool scan_by_token(int32_t total, int32_t max_seq) { return std::min(total, max_seq) <= kScanShort; }

// [tokens] rows of `cols` bf16 at a stride; boxes of 128 tokens x 64 columns
int map_bf16_strided(CUtensorMap* m, const void* base, int64_t tokens, int64_t cols,
                     int64_t stride) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return PHS_ECUDA;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(tokens)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride) * 2};
  cuuint32_t box[2] = {64, kScanChunk};
  cuuint32_t es[2] = {1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides,
                   box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? PHS_OK : PHS_ECUDA;
}

}  // namespace

extern "C" {

int phs_causal_conv_decode(const void* x, int64_t x_stride, const phs_conv_pool* pool,
                           const phs_conv_weights* weights, const int32_t* state_ids,
                           int32_t batch, void* out, int32_t* dev_status, void* stream) {
  ConvArgs a;
  const int st =
      conv_args(a, x, x_stride, pool, weights, state_ids, batch, batch, out, dev_status);
  if (st) return st;
  if (batch > 65535) return PHS_EUNSUPPORTED;  // grid y
  if (batch == 0) return PHS_OK;
  const int64_t channels = pool->channels;
  if (overlap_in_part({x, x_stride, channels, 2}, {out, channels, channels, 2}, batch))
    return PHS_EINVAL;
  return launch_conv_decode(pool->width, a, reinterpret_cast<cudaStream_t>(stream));
}

int phs_causal_conv_prompt(const void* x, int64_t x_stride, const int32_t* cu_seqlens,
                           int32_t total_tokens, const phs_conv_pool* pool,
                           const phs_conv_weights* weights, const int32_t* state_ids,
                           const int32_t* resume, int32_t batch, void* out, int32_t* dev_status,
                           void* stream) {
  ConvArgs a;
  int st =
      conv_args(a, x, x_stride, pool, weights, state_ids, batch, total_tokens, out, dev_status);
  if (st) return st;
  if (!cu_seqlens) return PHS_EINVAL;
  // (a tile's rows are read again, as earlier inputs, by the next one)
  const int64_t channels = pool->channels;
  if (overlap({x, x_stride, channels, 2}, {out, channels, channels, 2}, total_tokens))
    return PHS_EINVAL;
  if (batch == 0) return PHS_OK;
  a.cu_seqlens = cu_seqlens;
  a.resume = resume;
  DevInfo di;
  if ((st = dev_info(di))) return st;
  return launch_conv_prompt(pool->width, a, di.sms, reinterpret_cast<cudaStream_t>(stream));
}

int phs_selective_scan_decode(const phs_scan_inputs* in, const phs_scan_pool* pool,
                              const phs_scan_weights* weights, const int32_t* state_ids,
                              int32_t batch, void* out, int32_t out_dtype, int32_t* dev_status,
                              void* stream) {
  ScanArgs a;
  const int st = scan_args(a, in, pool, weights, state_ids, batch, batch, out, out_dtype,
                           dev_status);
  if (st || batch == 0) return st;
  if (scan_overlap(a, pool->head_dim, pool->state_dim, batch)) return PHS_EINVAL;
  return launch_scan_decode(pool->head_dim, pool->state_dim, a,
                            reinterpret_cast<cudaStream_t>(stream));
}

size_t phs_scan_prompt_workspace_bytes(int32_t batch, int32_t num_heads, int32_t num_groups,
                                       int32_t head_dim, int32_t state_dim, int32_t total_tokens,
                                       int32_t max_seq_len) {
  if (batch < 0 || total_tokens < 0 || max_seq_len < 0 || num_heads <= 0 || num_groups <= 0 ||
      num_heads % num_groups != 0 || (head_dim != 64 && head_dim != 128) ||
      (state_dim != 64 && state_dim != 128) || num_heads > 65535)
    return 0;
  if (scan_by_token(total_tokens, max_seq_len)) return 256;
  DevInfo di;
  if (dev_info(di)) return 0;
  return scan_plan(batch, num_heads, num_groups, head_dim, state_dim, total_tokens, max_seq_len,
                   di.sms)
      .need;
}

int phs_selective_scan_prompt(const phs_scan_inputs* in, const int32_t* cu_seqlens,
                              int32_t total_tokens, int32_t max_seq_len,
                              const phs_scan_pool* pool, const phs_scan_weights* weights,
                              const int32_t* state_ids, const int32_t* resume, int32_t batch,
                              void* out, void* workspace, size_t workspace_bytes,
                              int32_t* dev_status, void* stream) {
  ScanArgs a;
  int st = scan_args(a, in, pool, weights, state_ids, batch, total_tokens, out, PHS_OUT_BF16,
                     dev_status);
  if (st) return st;
  if (!cu_seqlens || max_seq_len < 0) return PHS_EINVAL;
  if (too_many(total_tokens, 0)) return PHS_EUNSUPPORTED;
  if (batch == 0) return PHS_OK;
  if ((st = check_workspace(workspace, workspace_bytes,
                            phs_scan_prompt_workspace_bytes(
                                batch, a.H, a.G, pool->head_dim, pool->state_dim, total_tokens,
                                max_seq_len))))
    return st;
  if (scan_overlap(a, pool->head_dim, pool->state_dim, total_tokens)) return PHS_EINVAL;
  a.cu_seqlens = cu_seqlens;
  a.resume = resume;
  a.total_tokens = total_tokens;
  a.max_seq = max_seq_len;
  const int P = pool->head_dim, N = pool->state_dim;
  if (scan_by_token(total_tokens, max_seq_len)) {
    a.short_len = kScanShort;
    return launch_scan_short(P, N, a, false, reinterpret_cast<cudaStream_t>(stream));
  }
  DevInfo di;
  if ((st = dev_info(di))) return st;
  const ScanPlan plan = scan_plan(batch, a.H, a.G, P, N, total_tokens, max_seq_len, di.sms);
  a.P = P;
  a.slots = plan.slots;
  a.units = plan.units;
  a.nseg = plan.nseg;
  a.nsub = plan.nsub;
  a.max_chunks = (std::min(total_tokens, max_seq_len) + kScanChunk - 1) / kScanChunk;
  const int64_t ctas = int64_t{batch} * a.units * a.nseg;
  // (grids: rows along x, tables and sums along y and z)
  if (ctas > INT32_MAX || batch > 65535 || a.units > 65535) return PHS_EUNSUPPORTED;
  a.longest_first = ctas > di.sms && batch > 1 && batch <= kScanSort;
  a.short_len = batch > 1 ? kScanShort : -1;
  char* ws = reinterpret_cast<char*>(workspace);
  a.tables = reinterpret_cast<float*>(ws);
  a.ws = reinterpret_cast<float*>(ws + plan.tables);
  a.ws_log = reinterpret_cast<float*>(ws + plan.tables + plan.sums);
  CUtensorMap tb, tc, tx, to;
  const int64_t hp = int64_t{a.H} * P, gn = int64_t{a.G} * N;
  if ((st = map_bf16_strided(&tb, a.b, total_tokens, gn, a.b_stride))) return st;
  if ((st = map_bf16_strided(&tc, a.c, total_tokens, gn, a.c_stride))) return st;
  if ((st = map_bf16_strided(&tx, a.x, total_tokens, hp, a.x_stride))) return st;
  if ((st = map_bf16_strided(&to, out, total_tokens, hp, hp))) return st;
  return launch_scan_prompt(N, tb, tc, tx, to, a, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
