"""paged_hybrid_sliding_gb300 -- decode attention over a hybrid paged KV
cache (a paged Full-attention pool plus per-request SWA ring buffers), KV
append and block-32 INT8 quantisation, as hand-written CUDA for sm_103a
behind the C ABI of include/phs.h.

This module only marshals torch tensors into the C ABI: every step runs in
the library's kernels.  Tensors must be CUDA, contiguous and of the dtype
stated; the stream defaults to torch's current stream.  Errors returned by
the library raise PhsError.
"""
from __future__ import annotations

import ctypes
import math
from dataclasses import dataclass

import torch

from . import _lib

__all__ = [
    "PhsError", "PagedPool", "RingPool", "Int8Pool", "Layer",
    "kv_append_paged", "kv_append_ring", "kv_quant_int8_block32",
    "decode_workspace_bytes", "decode_tokens_per_split",
    "attn_decode_full_paged", "attn_decode_full_paged_split", "attn_merge_splits",
    "attn_decode_full_paged_noalloc", "NOALLOC_SCRATCH_BYTES",
    "attn_decode_shared_prefix", "shared_prefix_workspace_bytes",
    "attn_decode_swa_ring", "attn_decode_hybrid_stack", "hybrid_stack_workspace_bytes",
    "attn_decode_hybrid_stack_fused", "hybrid_stack_fused_workspace_bytes",
    "hybrid_kv_tokens", "copy_d2d", "read_checksum", "copy_pages", "PageAllocator", "RadixTree",
    "window_safe_len", "swa_ring_save", "swa_ring_seed", "lib", "PAGE", "QBLOCK",
    "pages_free", "pages_fork", "pages_compact", "pages_fork_workspace_bytes",
    "pages_compact_workspace_bytes",
    "DiffWeights", "attn_decode_diff_paged", "diff_workspace_bytes",
    "StatePool", "linear_attn_decode", "linear_attn_prompt", "linear_prompt_workspace_bytes",
    "Rope", "rope_frequencies", "rope_rotate", "kv_write_paged", "kv_read_paged",
    "ConvPool", "ConvWeights", "causal_conv_decode", "causal_conv_prompt",
    "ScanPool", "ScanWeights", "selective_scan_decode", "selective_scan_prompt",
    "scan_prompt_workspace_bytes",
]

PAGE = 16
QBLOCK = 32
OUT_BF16, OUT_F32 = 0, 1
NOALLOC_SCRATCH_BYTES = 32 << 20


class PhsError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        msg = lib().phs_status_str(code).decode()
        super().__init__(f"{what}: {msg} ({code})")


def lib():
    return _lib._lib or _lib.load()


def _check(code: int, what: str):
    if code != 0:
        raise PhsError(code, what)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _need(t, dtype, name, dims=None):
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.is_cuda and t.is_contiguous() \
            and (dims is None or t.dim() == dims):
        return t
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dims is not None and t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dims, got {t.dim()}")
    return t


def _opt(t, dtype, name, dims=None):
    return None if t is None else _need(t, dtype, name, dims)


def _stream(stream):
    # the raw handle: making a Stream object for it costs a small call 3 us
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()) if stream is None \
        else stream.cuda_stream


def _out_code(dtype):
    if dtype == torch.bfloat16:
        return OUT_BF16
    if dtype == torch.float32:
        return OUT_F32
    raise ValueError("out dtype must be bfloat16 or float32")


@dataclass
class PagedPool:
    """Full-attention pool: k, v bf16 [num_pages, Hkv, 16, D]."""
    k: torch.Tensor
    v: torch.Tensor

    def c(self):
        k, v = self.k, self.v
        _need(k, torch.bfloat16, "pool.k", 4)
        _need(v, torch.bfloat16, "pool.v", 4)
        n, h, p, d = shape = k.shape
        if shape != v.shape:
            raise ValueError("pool.k and pool.v shapes differ")
        return _lib.PagedPoolC(k.data_ptr(), v.data_ptr(), n, p, h, d)

    @staticmethod
    def empty(num_pages, num_kv_heads, head_dim, device="cuda"):
        shape = (num_pages, num_kv_heads, PAGE, head_dim)
        return PagedPool(torch.empty(shape, dtype=torch.bfloat16, device=device),
                         torch.empty(shape, dtype=torch.bfloat16, device=device))


@dataclass
class RingPool:
    """SWA ring pool: k, v bf16 [num_rings, Hkv, W, D]."""
    k: torch.Tensor
    v: torch.Tensor

    def c(self):
        _need(self.k, torch.bfloat16, "ring.k", 4)
        _need(self.v, torch.bfloat16, "ring.v", 4)
        if self.k.shape != self.v.shape:
            raise ValueError("ring.k and ring.v shapes differ")
        n, h, w, d = self.k.shape
        return _lib.RingPoolC(self.k.data_ptr(), self.v.data_ptr(), n, w, h, d)

    @staticmethod
    def empty(num_rings, num_kv_heads, window, head_dim, device="cuda"):
        shape = (num_rings, num_kv_heads, window, head_dim)
        return RingPool(torch.empty(shape, dtype=torch.bfloat16, device=device),
                        torch.empty(shape, dtype=torch.bfloat16, device=device))


# Token held by byte p of a 16-token half of a stored V^T row (see Int8Pool).
VT_TOKEN = tuple(2 * (p >> 2) + (p & 1) + 8 * ((p >> 1) & 1) for p in range(16))


@dataclass
class Int8Pool:
    """INT8 pool in its stored form (each code x as the byte x + 128):
    k uint8 [num_qpages, Hkv, 32 tokens, D]; v uint8 [num_qpages, Hkv, 2,
    D, 16] (transposed per 16-token half; byte p of a row holds token
    VT_TOKEN[p] of its half); scales fp32 [num_qpages, Hkv]."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor

    def c(self):
        _need(self.k, torch.uint8, "int8.k", 4)
        _need(self.v, torch.uint8, "int8.v", 5)
        _need(self.k_scale, torch.float32, "int8.k_scale", 2)
        _need(self.v_scale, torch.float32, "int8.v_scale", 2)
        n, h, q, d = self.k.shape
        if q != QBLOCK or tuple(self.v.shape) != (n, h, 2, d, QBLOCK // 2) \
                or tuple(self.k_scale.shape) != (n, h) or tuple(self.v_scale.shape) != (n, h):
            raise ValueError("inconsistent INT8 pool shapes")
        return _lib.Int8PoolC(self.k.data_ptr(), self.v.data_ptr(), self.k_scale.data_ptr(),
                              self.v_scale.data_ptr(), n, h, d)

    def codes(self, pages=None):
        """The signed codes (int8) of all pages, or of the page ids in
        `pages`, both token-major [pages, Hkv, 32, D]: a view of the stored
        form for inspection, not used by the decode path."""
        k, v = self.k, self.v
        if pages is not None:
            k, v = k.index_select(0, pages), v.index_select(0, pages)
        # stored row 16 hf + p (half hf, byte p) holds token 16 hf + VT_TOKEN[p]
        order = torch.tensor([16 * hf + t for hf in range(2) for t in VT_TOKEN], device=v.device)
        inv = torch.empty_like(order)
        inv[order] = torch.arange(QBLOCK, device=v.device)
        rows = v.transpose(-1, -2).reshape(*v.shape[:2], QBLOCK, v.shape[3])  # [.., 16 hf + p, D]
        vt = rows.index_select(-2, inv)  # [.., token, D]
        return ((k.to(torch.int16) - 128).to(torch.int8),
                (vt.to(torch.int16) - 128).to(torch.int8).contiguous())

    @staticmethod
    def empty(num_qpages, num_kv_heads, head_dim, device="cuda"):
        return Int8Pool(
            torch.empty((num_qpages, num_kv_heads, QBLOCK, head_dim), dtype=torch.uint8,
                        device=device),
            torch.empty((num_qpages, num_kv_heads, 2, head_dim, QBLOCK // 2), dtype=torch.uint8,
                        device=device),
            torch.empty((num_qpages, num_kv_heads), dtype=torch.float32, device=device),
            torch.empty((num_qpages, num_kv_heads), dtype=torch.float32, device=device))


# ------------------------------------------------------------------ append --
def kv_append_paged(pool: PagedPool, k_new, v_new, block_table, seq_lens, page_refcount=None,
                    status=None, stream=None):
    """Write token seq_lens[b]-1 of every request into its page slot."""
    pc = pool.c()
    _need(k_new, torch.bfloat16, "k_new", 3)
    _need(v_new, torch.bfloat16, "v_new", 3)
    _need(block_table, torch.int32, "block_table", 2)
    _need(seq_lens, torch.int32, "seq_lens", 1)
    _opt(page_refcount, torch.int32, "page_refcount", 1)
    _opt(status, torch.int32, "status")
    _check(lib().phs_kv_append_paged(ctypes.byref(pc), _ptr(k_new), _ptr(v_new), _ptr(block_table),
                                     block_table.shape[1], _ptr(seq_lens), seq_lens.shape[0],
                                     _ptr(page_refcount), _ptr(status), _stream(stream)),
           "kv_append_paged")


def kv_append_ring(ring: RingPool, k_new, v_new, ring_pos, ring_ids=None, status=None,
                   stream=None):
    """Write the new token of every request into ring slot ring_pos[b]."""
    rc = ring.c()
    _need(k_new, torch.bfloat16, "k_new", 3)
    _need(v_new, torch.bfloat16, "v_new", 3)
    _need(ring_pos, torch.int32, "ring_pos", 1)
    _opt(ring_ids, torch.int32, "ring_ids", 1)
    _opt(status, torch.int32, "status")
    _check(lib().phs_kv_append_ring(ctypes.byref(rc), _ptr(k_new), _ptr(v_new), _ptr(ring_ids),
                                    _ptr(ring_pos), ring_pos.shape[0], _ptr(status),
                                    _stream(stream)), "kv_append_ring")


def kv_quant_int8_block32(src: PagedPool, src_block_table, dst: Int8Pool, dst_qtable,
                          first_qblock, num_qblocks, max_qblocks: int, status=None, stream=None):
    """Quantise 32-token blocks of the bf16 pages into INT8 codes + fp32 scales."""
    sc, dc = src.c(), dst.c()
    _need(src_block_table, torch.int32, "src_block_table", 2)
    _need(dst_qtable, torch.int32, "dst_qtable", 2)
    _need(first_qblock, torch.int32, "first_qblock", 1)
    _need(num_qblocks, torch.int32, "num_qblocks", 1)
    _opt(status, torch.int32, "status")
    _check(lib().phs_kv_quant_int8_block32(
        ctypes.byref(sc), _ptr(src_block_table), src_block_table.shape[1], ctypes.byref(dc),
        _ptr(dst_qtable), dst_qtable.shape[1], _ptr(first_qblock), _ptr(num_qblocks),
        int(max_qblocks), first_qblock.shape[0], _ptr(status), _stream(stream)),
        "kv_quant_int8_block32")


# ------------------------------------------------------------------ decode --
def decode_workspace_bytes(batch, num_q_heads, num_kv_heads, head_dim, max_seq_len,
                           tokens_per_split=0, has_int8=False) -> int:
    """Workspace bytes for a decode call; 0 if the shape is not supported."""
    return int(lib().phs_decode_workspace_bytes(batch, num_q_heads, num_kv_heads, head_dim,
                                                max_seq_len, tokens_per_split,
                                                int(bool(has_int8))))


def decode_tokens_per_split(batch, num_kv_heads, max_seq_len, tokens_per_split=0) -> int:
    t = lib().phs_decode_tokens_per_split(batch, num_kv_heads, max_seq_len, tokens_per_split)
    _check(min(int(t), 0), "decode_tokens_per_split")
    return int(t)


def _decode_args(q, pool, block_table, seq_lens, int8, qtable, qlens, out, out_dtype, status):
    _need(q, torch.bfloat16, "q", 3)
    pc = pool.c()
    _need(block_table, torch.int32, "block_table", 2)
    _need(seq_lens, torch.int32, "seq_lens", 1)
    ic = None
    if int8 is not None:
        ic = int8.c()
        _need(qtable, torch.int32, "qtable", 2)
        _need(qlens, torch.int32, "qlens", 1)
    B, Hq, D = q.shape
    if out is None:
        out = torch.empty((B, Hq, D), dtype=out_dtype, device=q.device)
    _need(out, out.dtype, "out", 3)
    _opt(status, torch.int32, "status")
    return pc, ic, out


def _append_args(k_new, v_new, page_refcount, B, Hkv, D):
    """Checks of a fused append's new tokens ([B, Hkv, D] bf16, both or
    neither) and page reference counts."""
    if (k_new is None) != (v_new is None):
        raise ValueError("k_new and v_new go together")
    if k_new is not None:
        for t, name in ((k_new, "k_new"), (v_new, "v_new")):
            _need(t, torch.bfloat16, name, 3)
            if tuple(t.shape) != (B, Hkv, D):
                raise ValueError(f"{name} must be [batch, Hkv, D]")
    _opt(page_refcount, torch.int32, "page_refcount", 1)


def _workspace(workspace, nbytes, device):
    if workspace is None:
        # a zero size means the library rejects the shape: let the call
        # report the precise status
        return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)
    _need(workspace, torch.uint8, "workspace", 1)
    return workspace


def attn_decode_full_paged(q, pool: PagedPool, block_table, seq_lens, max_seq_len: int,
                           softmax_scale=None, int8: Int8Pool | None = None, qtable=None,
                           qlens=None, tokens_per_split=0, out=None, out_dtype=torch.bfloat16,
                           workspace=None, k_new=None, v_new=None, page_refcount=None,
                           status=None, stream=None):
    """Split-KV decode over the paged pool (optionally INT8 below qlens[b]);
    returns out [B, Hq, D].  k_new / v_new ([B, Hkv, D] bf16): append token
    seq_lens[b] - 1 in the same call (as kv_append_paged with page_refcount,
    then this call)."""
    pc, ic, out = _decode_args(q, pool, block_table, seq_lens, int8, qtable, qlens, out,
                               out_dtype, status)
    B, Hq, D = q.shape
    _append_args(k_new, v_new, page_refcount, B, pool.k.shape[1], D)
    scale = 1.0 / math.sqrt(D) if softmax_scale is None else float(softmax_scale)
    need = decode_workspace_bytes(B, Hq, pool.k.shape[1], D, max_seq_len, tokens_per_split,
                                  int8 is not None)
    ws = _workspace(workspace, need, q.device)
    _check(lib().phs_attn_decode_full_paged(
        _ptr(q), Hq, ctypes.byref(pc), _ptr(block_table), block_table.shape[1], _ptr(seq_lens),
        int(max_seq_len), None if ic is None else ctypes.byref(ic), _ptr(qtable),
        0 if qtable is None else qtable.shape[1], _ptr(qlens), B, scale, int(tokens_per_split),
        _ptr(out), _out_code(out.dtype), _ptr(ws), ws.numel(), _ptr(k_new), _ptr(v_new),
        _ptr(page_refcount), _ptr(status), _stream(stream)), "attn_decode_full_paged")
    return out


def attn_decode_full_paged_noalloc(q, pool: PagedPool, block_table, seq_lens,
                                   max_seq_len: int, out, softmax_scale=None,
                                   int8: Int8Pool | None = None, qtable=None, qlens=None,
                                   tokens_per_split=0, status=None, stream=None):
    """Same as attn_decode_full_paged, for callers that cannot provide a
    workspace (a host framework that owns all device memory, an engine that
    has reserved nearly all of HBM, a loop that must not call cudaMalloc).
    The partials go to the library's built-in 32 MiB scratch per GPU; `out`
    must be given.  Calls that overlap on the GPU share that scratch and
    race, so serialise them.  Raises PhsError (PHS_ESCRATCH) when the
    request needs more scratch than that."""
    pc, ic, out = _decode_args(q, pool, block_table, seq_lens, int8, qtable, qlens, out,
                               out.dtype, status)
    B, Hq, D = q.shape
    scale = 1.0 / math.sqrt(D) if softmax_scale is None else float(softmax_scale)
    _check(lib().phs_attn_decode_full_paged_noalloc(
        _ptr(q), Hq, ctypes.byref(pc), _ptr(block_table), block_table.shape[1], _ptr(seq_lens),
        int(max_seq_len), None if ic is None else ctypes.byref(ic), _ptr(qtable),
        0 if qtable is None else qtable.shape[1], _ptr(qlens), B, scale, int(tokens_per_split),
        _ptr(out), _out_code(out.dtype), _ptr(status), _stream(stream)),
        "attn_decode_full_paged_noalloc")
    return out


def shared_prefix_workspace_bytes(batch, num_q_heads, num_kv_heads, head_dim, max_seq_len,
                                  shared_len) -> int:
    """Workspace bytes for attn_decode_shared_prefix; 0 if unsupported."""
    return int(lib().phs_shared_prefix_workspace_bytes(batch, num_q_heads, num_kv_heads,
                                                       head_dim, max_seq_len, shared_len))


def attn_decode_shared_prefix(q, pool: PagedPool, block_table, seq_lens, max_seq_len: int,
                              shared_len: int, softmax_scale=None, out=None,
                              out_dtype=torch.bfloat16, workspace=None, k_new=None, v_new=None,
                              page_refcount=None, status=None, stream=None):
    """Decode for a batch whose block tables all start with the same
    shared_len / 16 prefix pages: the prefix is attended once per KV head
    for all requests on the tensor cores, each request's own tokens by the
    split-KV kernel, then merged.  Same result as attn_decode_full_paged.
    k_new / v_new ([B, Hkv, D] bf16): append token seq_lens[b] - 1 in the
    same call (as kv_append_paged with page_refcount, then this call)."""
    pc, _, out = _decode_args(q, pool, block_table, seq_lens, None, None, None, out, out_dtype,
                              status)
    B, Hq, D = q.shape
    _append_args(k_new, v_new, page_refcount, B, pool.k.shape[1], D)
    scale = 1.0 / math.sqrt(D) if softmax_scale is None else float(softmax_scale)
    need = shared_prefix_workspace_bytes(B, Hq, pool.k.shape[1], D, max_seq_len, shared_len)
    ws = _workspace(workspace, need, q.device)
    _check(lib().phs_attn_decode_shared_prefix(
        _ptr(q), Hq, ctypes.byref(pc), _ptr(block_table), block_table.shape[1], _ptr(seq_lens),
        int(max_seq_len), B, int(shared_len), scale, _ptr(out), _out_code(out.dtype), _ptr(ws),
        ws.numel(), _ptr(k_new), _ptr(v_new), _ptr(page_refcount), _ptr(status), _stream(stream)),
        "attn_decode_shared_prefix")
    return out


def attn_decode_full_paged_split(q, pool: PagedPool, block_table, seq_lens, max_seq_len: int,
                                 workspace, out, softmax_scale=None, int8=None, qtable=None,
                                 qlens=None, tokens_per_split=0, k_new=None, v_new=None,
                                 page_refcount=None, status=None, stream=None):
    """Split phase only (see attn_merge_splits); k_new / v_new as for
    attn_decode_full_paged."""
    pc, ic, out = _decode_args(q, pool, block_table, seq_lens, int8, qtable, qlens, out,
                               out.dtype, status)
    B, Hq, D = q.shape
    _append_args(k_new, v_new, page_refcount, B, pool.k.shape[1], D)
    scale = 1.0 / math.sqrt(D) if softmax_scale is None else float(softmax_scale)
    _need(workspace, torch.uint8, "workspace", 1)
    _check(lib().phs_attn_decode_full_paged_split(
        _ptr(q), Hq, ctypes.byref(pc), _ptr(block_table), block_table.shape[1], _ptr(seq_lens),
        int(max_seq_len), None if ic is None else ctypes.byref(ic), _ptr(qtable),
        0 if qtable is None else qtable.shape[1], _ptr(qlens), B, scale, int(tokens_per_split),
        _ptr(out), _out_code(out.dtype), _ptr(workspace), workspace.numel(), _ptr(k_new),
        _ptr(v_new), _ptr(page_refcount), _ptr(status), _stream(stream)),
        "attn_decode_full_paged_split")
    return out


def attn_merge_splits(out, num_kv_heads, seq_lens, max_seq_len: int, workspace, qlens=None,
                      has_int8=False, tokens_per_split=0, stream=None):
    """Merge phase only: finishes requests that the split phase cut in pieces."""
    B, Hq, D = out.shape
    _need(seq_lens, torch.int32, "seq_lens", 1)
    _opt(qlens, torch.int32, "qlens", 1)
    _need(workspace, torch.uint8, "workspace", 1)
    _check(lib().phs_attn_merge_splits(B, Hq, num_kv_heads, D, _ptr(seq_lens), int(max_seq_len),
                                       _ptr(qlens), int(bool(has_int8)), int(tokens_per_split),
                                       _ptr(out), _out_code(out.dtype), _ptr(workspace),
                                       workspace.numel(), _stream(stream)), "attn_merge_splits")
    return out


def attn_decode_swa_ring(q, ring: RingPool, ring_pos, seq_lens, ring_ids=None,
                         softmax_scale=None, out=None, out_dtype=torch.bfloat16, status=None,
                         stream=None):
    """Sliding-window decode over each request's ring; returns out [B, Hq, D]."""
    _need(q, torch.bfloat16, "q", 3)
    rc = ring.c()
    _need(ring_pos, torch.int32, "ring_pos", 1)
    _need(seq_lens, torch.int32, "seq_lens", 1)
    _opt(ring_ids, torch.int32, "ring_ids", 1)
    _opt(status, torch.int32, "status")
    B, Hq, D = q.shape
    if out is None:
        out = torch.empty((B, Hq, D), dtype=out_dtype, device=q.device)
    _need(out, out.dtype, "out", 3)
    scale = 1.0 / math.sqrt(D) if softmax_scale is None else float(softmax_scale)
    _check(lib().phs_attn_decode_swa_ring(_ptr(q), Hq, ctypes.byref(rc), _ptr(ring_ids),
                                          _ptr(ring_pos), _ptr(seq_lens), B, scale, _ptr(out),
                                          _out_code(out.dtype), _ptr(status), _stream(stream)),
           "attn_decode_swa_ring")
    return out


@dataclass
class Layer:
    """One layer of a hybrid stack: Full (paged pool) or SWA (ring pool)."""
    q: torch.Tensor
    out: torch.Tensor
    paged: PagedPool | None = None
    ring: RingPool | None = None
    k_new: torch.Tensor | None = None
    v_new: torch.Tensor | None = None

    def c(self):
        L = _lib.LayerC()
        L.is_full = 1 if self.paged is not None else 0
        L.q = self.q.data_ptr()
        L.out = self.out.data_ptr()
        L.k_new = 0 if self.k_new is None else self.k_new.data_ptr()
        L.v_new = 0 if self.v_new is None else self.v_new.data_ptr()
        if self.paged is not None:
            L.paged = self.paged.c()
        else:
            L.ring = self.ring.c()
        return L


def hybrid_stack_workspace_bytes(batch, num_q_heads, num_kv_heads, head_dim, max_seq_len):
    return int(lib().phs_hybrid_stack_workspace_bytes(batch, num_q_heads, num_kv_heads, head_dim,
                                                      max_seq_len))


def attn_decode_hybrid_stack(layers, num_q_heads, seq_lens, max_seq_len, block_table=None,
                             ring_pos=None, ring_ids=None, softmax_scale=None, do_append=True,
                             workspace=None, status=None, stream=None, page_refcount=None):
    """One decode step (append + attend) over every layer of a hybrid stack.
    page_refcount: optional device int32 [num_pages]; a Full layer's new token
    is not written into a page whose count is not 1."""
    arr = (_lib.LayerC * len(layers))(*[L.c() for L in layers])
    _need(seq_lens, torch.int32, "seq_lens", 1)
    _opt(block_table, torch.int32, "block_table", 2)
    _opt(page_refcount, torch.int32, "page_refcount", 1)
    _opt(ring_pos, torch.int32, "ring_pos", 1)
    _opt(ring_ids, torch.int32, "ring_ids", 1)
    _opt(status, torch.int32, "status")
    B = seq_lens.shape[0]
    q0 = layers[0].q
    D = q0.shape[2]
    out_code = _out_code(layers[0].out.dtype)
    scale = 1.0 / math.sqrt(D) if softmax_scale is None else float(softmax_scale)
    nfull = sum(1 for L in layers if L.paged is not None)
    if workspace is None and nfull:
        hkv = next(L.paged.k.shape[1] for L in layers if L.paged is not None)
        workspace = torch.empty(hybrid_stack_workspace_bytes(B, num_q_heads, hkv, D, max_seq_len),
                                dtype=torch.uint8, device=q0.device)
    _check(lib().phs_attn_decode_hybrid_stack(
        arr, len(layers), num_q_heads, B, _ptr(block_table),
        0 if block_table is None else block_table.shape[1], _ptr(page_refcount),
        _ptr(seq_lens), int(max_seq_len),
        _ptr(ring_ids), _ptr(ring_pos), scale, int(bool(do_append)), out_code, _ptr(workspace),
        0 if workspace is None else workspace.numel(), _ptr(status), _stream(stream)),
        "attn_decode_hybrid_stack")


def hybrid_stack_fused_workspace_bytes(batch, num_q_heads, num_kv_heads, head_dim, max_seq_len,
                                       num_full_layers):
    return int(lib().phs_hybrid_stack_fused_workspace_bytes(batch, num_q_heads, num_kv_heads,
                                                            head_dim, max_seq_len,
                                                            num_full_layers))


def attn_decode_hybrid_stack_fused(layers, num_q_heads, seq_lens, max_seq_len, block_table=None,
                                   ring_pos=None, ring_ids=None, softmax_scale=None,
                                   workspace=None, status=None, stream=None, page_refcount=None):
    """One decode step over every layer of a hybrid stack with the appends
    fused into the attention launches (every layer needs k_new / v_new).
    page_refcount as for attn_decode_hybrid_stack."""
    arr = (_lib.LayerC * len(layers))(*[L.c() for L in layers])
    _need(seq_lens, torch.int32, "seq_lens", 1)
    _opt(block_table, torch.int32, "block_table", 2)
    _opt(page_refcount, torch.int32, "page_refcount", 1)
    _opt(ring_pos, torch.int32, "ring_pos", 1)
    _opt(ring_ids, torch.int32, "ring_ids", 1)
    _opt(status, torch.int32, "status")
    B = seq_lens.shape[0]
    q0 = layers[0].q
    D = q0.shape[2]
    out_code = _out_code(layers[0].out.dtype)
    scale = 1.0 / math.sqrt(D) if softmax_scale is None else float(softmax_scale)
    nfull = sum(1 for L in layers if L.paged is not None)
    if workspace is None and nfull:
        hkv = next(L.paged.k.shape[1] for L in layers if L.paged is not None)
        workspace = torch.empty(hybrid_stack_fused_workspace_bytes(B, num_q_heads, hkv, D,
                                                                   max_seq_len, nfull),
                                dtype=torch.uint8, device=q0.device)
    _check(lib().phs_attn_decode_hybrid_stack_fused(
        arr, len(layers), num_q_heads, B, _ptr(block_table),
        0 if block_table is None else block_table.shape[1], _ptr(page_refcount),
        _ptr(seq_lens), int(max_seq_len),
        _ptr(ring_ids), _ptr(ring_pos), scale, out_code, _ptr(workspace),
        0 if workspace is None else workspace.numel(), _ptr(status), _stream(stream)),
        "attn_decode_hybrid_stack_fused")


def hybrid_kv_tokens(layer_is_full, seq_lens_host, window):
    """(Full-layer tokens, SWA-layer tokens) held by a stack; host lists in."""
    import numpy as np
    lf = np.ascontiguousarray(layer_is_full, dtype=np.int32)
    sl = np.ascontiguousarray(seq_lens_host, dtype=np.int32)
    f, w = ctypes.c_int64(), ctypes.c_int64()
    _check(lib().phs_hybrid_kv_tokens(lf.ctypes.data, lf.shape[0], sl.ctypes.data, sl.shape[0],
                                      int(window), ctypes.byref(f), ctypes.byref(w)),
           "hybrid_kv_tokens")
    return f.value, w.value


def copy_d2d(dst, src, stream=None):
    """HBM copy kernel: dst <- src (same byte size, 16-byte multiples)."""
    if dst.numel() * dst.element_size() != src.numel() * src.element_size():
        raise ValueError("copy_d2d size mismatch")
    _check(lib().phs_copy_d2d(_ptr(dst), _ptr(src), src.numel() * src.element_size(),
                              _stream(stream)), "copy_d2d")


def read_checksum(src, sink, stream=None):
    """HBM read kernel: XOR every 32-bit word of `src` (contiguous, a
    multiple of 16 bytes) into sink[0] (CUDA int32 tensor, not cleared)."""
    _need(sink, torch.int32, "sink")
    if not src.is_contiguous():
        raise ValueError("src must be contiguous")
    _check(lib().phs_read_checksum(_ptr(src), src.numel() * src.element_size(), _ptr(sink),
                                   _stream(stream)), "read_checksum")


# ------------------------------------------------------- cache bookkeeping --
def copy_pages(pool: PagedPool, src_pages, dst_pages, status=None, stream=None):
    """Device copy of whole pages (K and V): dst_pages[i] <- src_pages[i]."""
    pc = pool.c()
    _need(src_pages, torch.int32, "src_pages", 1)
    _need(dst_pages, torch.int32, "dst_pages", 1)
    _opt(status, torch.int32, "status")
    _check(lib().phs_copy_pages(ctypes.byref(pc), _ptr(src_pages), _ptr(dst_pages),
                                src_pages.shape[0], _ptr(status), _stream(stream)), "copy_pages")


def _i32(a):
    import numpy as np
    return np.ascontiguousarray(a, dtype=np.int32)


class PageAllocator:
    """Refcounted page allocator (host object of the library)."""

    def __init__(self, num_pages: int):
        self.num_pages = int(num_pages)
        self._h = lib().phs_page_allocator_create(self.num_pages)
        if not self._h:
            raise ValueError("bad number of pages")

    def close(self):
        if self._h:
            lib().phs_page_allocator_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def alloc(self, n: int):
        import numpy as np
        out = np.empty(max(int(n), 0), dtype=np.int32)
        _check(lib().phs_page_alloc(self._h, int(n), out.ctypes.data), "page_alloc")
        return out

    def incref(self, pages):
        p = _i32(pages)
        _check(lib().phs_page_incref(self._h, p.ctypes.data, p.shape[0]), "page_incref")

    def decref(self, pages):
        p = _i32(pages)
        _check(lib().phs_page_decref(self._h, p.ctypes.data, p.shape[0]), "page_decref")

    def free_count(self) -> int:
        return int(lib().phs_page_free_count(self._h))

    def refcounts(self):
        import numpy as np
        out = np.empty(self.num_pages, dtype=np.int32)
        _check(lib().phs_page_refcounts(self._h, out.ctypes.data), "page_refcounts")
        return out

    def load_refcounts(self, counts):
        """Take counts (host int32 [num_pages]) as the allocator's own: what
        pages_free / pages_fork / pages_compact left on the device."""
        c = _i32(counts)
        if c.shape != (self.num_pages,):
            raise ValueError("counts must be [num_pages]")
        _check(lib().phs_page_load_refcounts(self._h, c.ctypes.data), "page_load_refcounts")

    def cow(self, page: int) -> int:
        out = ctypes.c_int32()
        _check(lib().phs_page_cow(self._h, int(page), ctypes.byref(out)), "page_cow")
        return out.value


class RadixTree:
    """Radix prefix tree over whole pages, holding references in `alloc`
    (Full pages) and `swa_alloc` (SWA segment pages, optional)."""

    def __init__(self, alloc: PageAllocator, page_size: int = PAGE,
                 swa_alloc: PageAllocator | None = None):
        self.alloc = alloc
        self.swa_alloc = swa_alloc
        self.page_size = int(page_size)
        self._h = lib().phs_radix_create(alloc._h, None if swa_alloc is None else swa_alloc._h,
                                         self.page_size)
        if not self._h:
            raise ValueError("bad radix tree arguments")

    def close(self):
        if self._h:
            lib().phs_radix_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def match(self, tokens):
        """Matched page ids (each gets a reference for the caller)."""
        import numpy as np
        t = _i32(tokens)
        cap = t.shape[0] // self.page_size + 1
        out = np.empty(cap, dtype=np.int32)
        n = ctypes.c_int32()
        _check(lib().phs_radix_match(self._h, t.ctypes.data, t.shape[0], out.ctypes.data, cap,
                                     ctypes.byref(n)), "radix_match")
        return out[:n.value].copy()

    def match_window_safe(self, tokens, window: int):
        """(Full pages, SWA segment pages of the last window) of the longest
        window-safe match; each id gets a reference for the caller."""
        import numpy as np
        t = _i32(tokens)
        cap = t.shape[0] // self.page_size + 1
        out = np.empty(cap, dtype=np.int32)
        seg = np.empty(cap, dtype=np.int32)
        n, ns = ctypes.c_int32(), ctypes.c_int32()
        _check(lib().phs_radix_match_window_safe(self._h, t.ctypes.data, t.shape[0], int(window),
                                                 out.ctypes.data, cap, ctypes.byref(n),
                                                 seg.ctypes.data, cap, ctypes.byref(ns)),
               "radix_match_window_safe")
        return out[:n.value].copy(), seg[:ns.value].copy()

    def insert(self, tokens, pages, swa_pages=None):
        """Cache the whole pages of `tokens`; swa_pages: per page, the SWA
        segment page holding its SWA-layer KV, or -1 (None: none)."""
        t, p = _i32(tokens), _i32(pages)
        s = None if swa_pages is None else _i32(swa_pages)
        if s is not None and s.shape[0] < t.shape[0] // self.page_size:
            raise ValueError("swa_pages needs one entry per whole page")
        _check(lib().phs_radix_insert(self._h, t.ctypes.data, t.shape[0], p.ctypes.data,
                                      None if s is None else s.ctypes.data), "radix_insert")

    def evict(self, pages: int) -> int:
        freed = ctypes.c_int64()
        _check(lib().phs_radix_evict(self._h, int(pages), ctypes.byref(freed)), "radix_evict")
        return freed.value

    def remap(self, page_map):
        """Rename the tree's Full pages by the map pages_compact wrote (host
        int32 [num_pages])."""
        m = _i32(page_map)
        _check(lib().phs_radix_remap(self._h, m.ctypes.data, m.shape[0]), "radix_remap")

    def cached_pages(self) -> int:
        return int(lib().phs_radix_cached_pages(self._h))


def _pool_array(ctype, pools):
    return (ctype * len(pools))(*[p.c() for p in pools])


def swa_ring_save(rings, segs, ring_ids, ring_pos, seq_lens, page_index, seg_pages, status=None,
                  stream=None):
    """Snapshot whole pages of requests' SWA windows into segment pages, in
    every SWA layer: entry i copies logical page page_index[i] of the
    request with ring ring_ids[i] (newest slot ring_pos[i], length
    seq_lens[i]) into segment page seg_pages[i].  rings: list of RingPool,
    segs: list of PagedPool (one per SWA layer)."""
    if len(rings) != len(segs) or not rings:
        raise ValueError("one segment pool per ring pool")
    for name, t in (("ring_ids", ring_ids), ("ring_pos", ring_pos), ("seq_lens", seq_lens),
                    ("page_index", page_index), ("seg_pages", seg_pages)):
        _need(t, torch.int32, name, 1)
    _opt(status, torch.int32, "status")
    _check(lib().phs_swa_ring_save(_pool_array(_lib.RingPoolC, rings),
                                   _pool_array(_lib.PagedPoolC, segs), len(rings),
                                   _ptr(ring_ids), _ptr(ring_pos), _ptr(seq_lens),
                                   _ptr(page_index), _ptr(seg_pages), page_index.shape[0],
                                   _ptr(status), _stream(stream)), "swa_ring_save")


def swa_ring_seed(rings, segs, ring_pos, seq_lens, seg_table, ring_ids=None, status=None,
                  stream=None):
    """Fill each request's ring, in every SWA layer, with the last
    min(n, W) tokens from the segment pages of its row of seg_table
    ([B, max_seg] int32), newest token at slot ring_pos[b]."""
    if len(rings) != len(segs) or not rings:
        raise ValueError("one segment pool per ring pool")
    _need(ring_pos, torch.int32, "ring_pos", 1)
    _need(seq_lens, torch.int32, "seq_lens", 1)
    _need(seg_table, torch.int32, "seg_table", 2)
    _opt(ring_ids, torch.int32, "ring_ids", 1)
    _opt(status, torch.int32, "status")
    _check(lib().phs_swa_ring_seed(_pool_array(_lib.RingPoolC, rings),
                                   _pool_array(_lib.PagedPoolC, segs), len(rings),
                                   _ptr(ring_ids), _ptr(ring_pos), _ptr(seq_lens),
                                   _ptr(seg_table), seg_table.shape[1], seq_lens.shape[0],
                                   _ptr(status), _stream(stream)), "swa_ring_seed")


def window_safe_len(swa_valid, match_len: int, window: int, align: int = 1) -> int:
    import numpy as np
    v = np.ascontiguousarray(swa_valid, dtype=np.uint8)
    r = int(lib().phs_window_safe_len(v.ctypes.data, int(match_len), int(window), int(align)))
    _check(min(r, 0), "window_safe_len")
    return r


# ---------------------------------------------------------- page operations --
# A small call costs the GPU less than its checks cost the host, so the calls
# below look at each tensor once.
_DEVICE_ERROR = "all tensors must be on the current CUDA device"


def _device(t, dtype, name):
    """The device that a call with t runs on: t's, and the current one."""
    if isinstance(t, torch.Tensor):
        dev = t.get_device()
        if dev >= 0:
            if torch._C._cuda_getDevice() != dev:
                raise ValueError(_DEVICE_ERROR)
            return dev
    return _need(t, dtype, name).get_device()


def _shape(t, dtype, dev, name, dims):
    """Shape of t: a contiguous `dtype` tensor of `dims` dimensions on `dev`."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev \
            and t.is_contiguous():
        shape = t.shape
        if len(shape) == dims:
            return shape
    _need(t, dtype, name, dims)
    raise ValueError(_DEVICE_ERROR)


def _status_ptr(status, dev):
    if status is None:
        return None
    if _need(status, torch.int32, "status").get_device() != dev:
        raise ValueError(_DEVICE_ERROR)
    return status.data_ptr()


def _raw_stream(stream, dev):
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


_devices: dict[int, torch.device] = {}  # (made once: torch takes 0.7 us to make one of an index)


def _empty(shape, dtype, device, stream):
    """Memory for a call on `stream` (None: the current one), from that
    stream's own: what the current stream has let go of may still be in use
    there, and what this call uses must not be handed on before it is done."""
    d = _devices.get(device)
    if d is None:
        d = _devices[device] = torch.device("cuda", device)
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=d)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=d)


def _call_memory(workspace, nbytes, dev, stream):
    """(pointer, bytes) of a call's workspace, and the tensor that holds it."""
    if workspace is None:
        # (a zero size means the library rejects the shape: it says how)
        workspace = _empty((max(nbytes, 1),), torch.uint8, dev, stream)
        return workspace.data_ptr(), nbytes, workspace
    n, = _shape(workspace, torch.uint8, dev, "workspace", 1)
    return workspace.data_ptr(), n, workspace


def _tables(block_table, seq_lens, page_refcount):
    """(device, rows, pages of a row, pages of the pool)"""
    dev = _device(block_table, torch.int32, "block_table")
    rows, width = _shape(block_table, torch.int32, dev, "block_table", 2)
    n, = _shape(seq_lens, torch.int32, dev, "seq_lens", 1)
    pages, = _shape(page_refcount, torch.int32, dev, "page_refcount", 1)
    if n != rows:
        raise ValueError("seq_lens needs one entry per row of block_table")
    return dev, rows, width, pages


def _pool_c(pool, dev):
    shape = n, h, p, d = _shape(pool.k, torch.bfloat16, dev, "pool.k", 4)
    if _shape(pool.v, torch.bfloat16, dev, "pool.v", 4) != shape:
        raise ValueError("pool.k and pool.v shapes differ")
    return _lib.PagedPoolC(pool.k.data_ptr(), pool.v.data_ptr(), n, p, h, d)


def _pools_of(pools, dev, num_pages):
    if not pools:
        raise ValueError("pools must name at least one pool")
    arr = (_lib.PagedPoolC * len(pools))()
    for i, p in enumerate(pools):
        arr[i] = c = _pool_c(p, dev)
        if c.num_pages != num_pages:
            raise ValueError("page_refcount needs one entry per page")
    return arr


def pages_free(block_table, seq_lens, page_refcount, rows, status=None, stream=None):
    """Free the listed rows of the block table: one reference less on each
    of their pages, their lengths zero."""
    dev, num_rows, width, pages = _tables(block_table, seq_lens, page_refcount)
    n, = _shape(rows, torch.int32, dev, "rows", 1)
    _check(lib().phs_pages_free(block_table.data_ptr(), num_rows, width, seq_lens.data_ptr(),
                                page_refcount.data_ptr(), pages, rows.data_ptr(), n,
                                _status_ptr(status, dev), _raw_stream(stream, dev)),
           "pages_free")


def pages_fork_workspace_bytes(num_rows, n) -> int:
    return int(lib().phs_pages_fork_workspace_bytes(num_rows, n))


def pages_fork(pools, block_table, seq_lens, page_refcount, src_rows, dst_rows, workspace=None,
               status=None, stream=None):
    """Continue row src_rows[i] in the free row dst_rows[i]: whole pages
    shared, a partly filled last page copied into the lowest free page, in
    every pool of `pools` (list of PagedPool sharing the block table).  Pages
    of the block table only: an INT8 region, SWA rings and linear attention
    states are the caller's to copy."""
    dev, rows, width, pages = _tables(block_table, seq_lens, page_refcount)
    n, = _shape(src_rows, torch.int32, dev, "src_rows", 1)
    if _shape(dst_rows, torch.int32, dev, "dst_rows", 1) != (n,):
        raise ValueError("src_rows and dst_rows go together")
    arr = _pools_of(pools, dev, pages)
    ws, ws_bytes, _held = _call_memory(workspace, pages_fork_workspace_bytes(rows, n), dev, stream)
    _check(lib().phs_pages_fork(arr, len(pools), block_table.data_ptr(), rows, width,
                                seq_lens.data_ptr(), page_refcount.data_ptr(),
                                src_rows.data_ptr(), dst_rows.data_ptr(), n, ws, ws_bytes,
                                _status_ptr(status, dev), _raw_stream(stream, dev)),
           "pages_fork")


def pages_compact_workspace_bytes(num_pages) -> int:
    return int(lib().phs_pages_compact_workspace_bytes(num_pages))


def pages_compact(pools, block_table, seq_lens, page_refcount, block_table_out=None,
                  page_refcount_out=None, page_map=None, num_live=None, workspace=None,
                  status=None, stream=None):
    """Move the live pages to the lowest page ids in every pool of `pools`;
    returns (page_map [num_pages]: new id or -1, num_live [1]).  The tables
    and counts are rewritten in place unless *_out are given."""
    dev, rows, width, pages = _tables(block_table, seq_lens, page_refcount)
    arr = _pools_of(pools, dev, pages)
    bt = block_table if block_table_out is None else block_table_out
    rc = page_refcount if page_refcount_out is None else page_refcount_out
    if page_map is None:
        page_map = _empty((pages,), torch.int32, dev, stream)
    if num_live is None:
        num_live = _empty((1,), torch.int32, dev, stream)
    if bt is not block_table and \
            _shape(bt, torch.int32, dev, "block_table_out", 2) != (rows, width):
        raise ValueError(f"block_table_out must be [{rows}, {width}]")
    if rc is not page_refcount and \
            _shape(rc, torch.int32, dev, "page_refcount_out", 1) != (pages,):
        raise ValueError(f"page_refcount_out must be [{pages}]")
    if _shape(page_map, torch.int32, dev, "page_map", 1) != (pages,):
        raise ValueError(f"page_map must be [{pages}]")
    if _shape(num_live, torch.int32, dev, "num_live", 1) != (1,):
        raise ValueError("num_live must be [1]")
    ws, ws_bytes, _held = _call_memory(workspace, pages_compact_workspace_bytes(pages), dev, stream)
    _check(lib().phs_pages_compact(arr, len(pools), block_table.data_ptr(), rows, width,
                                   seq_lens.data_ptr(), page_refcount.data_ptr(), bt.data_ptr(),
                                   rc.data_ptr(), page_map.data_ptr(), num_live.data_ptr(), ws,
                                   ws_bytes, _status_ptr(status, dev), _raw_stream(stream, dev)),
           "pages_compact")
    return page_map, num_live


# --------------------------------------------------- differential attention --
@dataclass
class DiffWeights:
    """Learned weights of a differential attention layer: lambda vectors
    fp32 [D] (or [H, D], one per head) and, for the norm of each head's
    output, fp32 [2D] (None: no norm)."""
    lambda_q1: torch.Tensor
    lambda_k1: torch.Tensor
    lambda_q2: torch.Tensor
    lambda_k2: torch.Tensor
    lambda_init: float
    norm_weight: torch.Tensor | None = None
    norm_eps: float = 1e-5

    def c(self, num_heads, head_dim, dev):
        per_head = self.lambda_q1.dim() == 2
        want = (num_heads, head_dim) if per_head else (head_dim,)
        vecs = (self.lambda_q1, self.lambda_k1, self.lambda_q2, self.lambda_k2)
        for t in vecs:
            if _shape(t, torch.float32, dev, "lambda vectors", len(want)) != want:
                raise ValueError(f"lambda vectors must be [{head_dim}] or "
                                 f"[{num_heads}, {head_dim}], all alike")
        norm = self.norm_weight
        if norm is not None and \
                _shape(norm, torch.float32, dev, "norm_weight", 1) != (2 * head_dim,):
            raise ValueError(f"norm_weight must be [{2 * head_dim}]")
        return _lib.DiffWeightsC(*[t.data_ptr() for t in vecs], _ptr(norm),
                                 float(self.lambda_init), float(self.norm_eps), per_head)


def diff_workspace_bytes(batch, num_heads, num_value_heads, head_dim, max_seq_len,
                         tokens_per_split=0) -> int:
    """Workspace bytes for attn_decode_diff_paged; 0 if unsupported."""
    return int(lib().phs_diff_workspace_bytes(batch, num_heads, num_value_heads, head_dim,
                                              max_seq_len, tokens_per_split))


def attn_decode_diff_paged(q, pool: PagedPool, block_table, seq_lens, max_seq_len: int,
                           weights: DiffWeights, softmax_scale=None, tokens_per_split=0, out=None,
                           out_dtype=torch.bfloat16, workspace=None, k_new=None, v_new=None,
                           page_refcount=None, status=None, stream=None):
    """Differential attention decode: q [B, 2H, D] (rows 2i, 2i + 1: head i's
    queries of the two maps), pool of 2 Hv heads of width D; returns out
    [B, H, 2D].  k_new / v_new ([B, 2 Hv, D] bf16): append token
    seq_lens[b] - 1 in the same call."""
    dev = _device(q, torch.bfloat16, "q")
    B, H2, D = _shape(q, torch.bfloat16, dev, "q", 3)
    pc = _pool_c(pool, dev)
    rows, width = _shape(block_table, torch.int32, dev, "block_table", 2)
    n, = _shape(seq_lens, torch.int32, dev, "seq_lens", 1)
    heads = pc.num_kv_heads
    if H2 % 2 != 0 or heads % 2 != 0:
        raise ValueError("q and the pool need an even number of heads (two maps)")
    if D != pc.head_dim:
        raise ValueError("q and the pool differ in head_dim")
    if rows != B or n != B:
        raise ValueError("block_table and seq_lens need one row per request")
    H = H2 // 2
    if out is None:
        out = _empty((B, H, 2 * D), out_dtype, dev, stream)
    elif _shape(out, out.dtype, dev, "out", 3) != (B, H, 2 * D):
        raise ValueError("out must be [batch, H, 2 head_dim]")
    if (k_new is None) != (v_new is None):
        raise ValueError("k_new and v_new go together")
    if k_new is not None and (_shape(k_new, torch.bfloat16, dev, "k_new", 3) != (B, heads, D) or
                              _shape(v_new, torch.bfloat16, dev, "v_new", 3) != (B, heads, D)):
        raise ValueError("k_new and v_new must be [batch, heads of the pool, D]")
    if page_refcount is not None and \
            _shape(page_refcount, torch.int32, dev, "page_refcount", 1) != (pc.num_pages,):
        raise ValueError("page_refcount needs one entry per page")
    wc = weights.c(H, D, dev)
    scale = 1.0 / math.sqrt(D) if softmax_scale is None else float(softmax_scale)
    ws, ws_bytes, _held = _call_memory(
        workspace, diff_workspace_bytes(B, H, heads // 2, D, max_seq_len, tokens_per_split), dev,
        stream)
    _check(lib().phs_attn_decode_diff_paged(
        q.data_ptr(), H, pc, block_table.data_ptr(), width, seq_lens.data_ptr(), int(max_seq_len),
        B, wc, scale, int(tokens_per_split), out.data_ptr(), _out_code(out.dtype), ws, ws_bytes,
        _ptr(k_new), _ptr(v_new), _ptr(page_refcount), _status_ptr(status, dev),
        _raw_stream(stream, dev)), "attn_decode_diff_paged")
    return out


# --------------------------------------------------------- linear attention --
@dataclass
class StatePool:
    """States of linear attention: s fp32 [num_states, Hkv, D (k), D (v)]."""
    s: torch.Tensor

    def c(self, dev):
        n, h, d, d2 = _shape(self.s, torch.float32, dev, "state.s", 4)
        if d != d2:
            raise ValueError("state.s must be [num_states, Hkv, D, D]")
        return _lib.StatePoolC(self.s.data_ptr(), n, h, d)

    @staticmethod
    def zeros(num_states, num_kv_heads, head_dim, device="cuda"):
        return StatePool(torch.zeros((num_states, num_kv_heads, head_dim, head_dim),
                                     dtype=torch.float32, device=device))


def _linear_args(q, k, v, pool, log_decay, state_ids, batch, dev):
    """(T, Hq, D) of q and the pool's descriptor, all arguments checked."""
    T, Hq, D = _shape(q, torch.bfloat16, dev, "q", 3)
    pc = pool.c(dev)
    Hkv = pc.num_kv_heads
    if _shape(k, torch.bfloat16, dev, "k", 3) != (T, Hkv, D) or \
            _shape(v, torch.bfloat16, dev, "v", 3) != (T, Hkv, D):
        raise ValueError("k and v must be [tokens, Hkv, head_dim]")
    if D != pc.head_dim:
        raise ValueError("q and the state pool differ in head_dim")
    if _shape(log_decay, torch.float32, dev, "log_decay", 1) != (Hkv,):
        raise ValueError("log_decay must be [Hkv]")
    batch = T if batch is None else batch
    if state_ids is not None and \
            _shape(state_ids, torch.int32, dev, "state_ids", 1) != (batch,):
        raise ValueError("state_ids must be [batch]")
    return T, Hq, D, pc


def _linear_out(out, T, Hq, D, dtype, dev, stream):
    if out is None:
        return _empty((T, Hq, D), dtype, dev, stream)
    if _shape(out, out.dtype, dev, "out", 3) != (T, Hq, D):
        raise ValueError("out must have q's shape")
    return out


def linear_attn_decode(q, k_new, v_new, pool: StatePool, log_decay, state_ids=None, scale=None,
                       out=None, out_dtype=torch.bfloat16, status=None, stream=None):
    """One token of linear attention per request: q [B, Hq, D], k_new, v_new
    [B, Hkv, D] bf16; updates the states and returns out [B, Hq, D]."""
    dev = _device(q, torch.bfloat16, "q")
    B, Hq, D, pc = _linear_args(q, k_new, v_new, pool, log_decay, state_ids, None, dev)
    out = _linear_out(out, B, Hq, D, out_dtype, dev, stream)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    _check(lib().phs_linear_attn_decode(q.data_ptr(), Hq, pc, k_new.data_ptr(), v_new.data_ptr(),
                                        log_decay.data_ptr(), _ptr(state_ids), B, scale,
                                        out.data_ptr(), _out_code(out.dtype),
                                        _status_ptr(status, dev), _raw_stream(stream, dev)),
           "linear_attn_decode")
    return out


def linear_prompt_workspace_bytes(batch, num_q_heads, num_kv_heads, head_dim, total_tokens,
                                  max_seq_len) -> int:
    """Workspace bytes for linear_attn_prompt; 0 if unsupported.  For a call
    of these very sizes: one with fewer requests may need more."""
    return int(lib().phs_linear_prompt_workspace_bytes(batch, num_q_heads, num_kv_heads, head_dim,
                                                       total_tokens, max_seq_len))


def linear_attn_prompt(q, k, v, cu_seqlens, max_seq_len: int, pool: StatePool, log_decay,
                       state_ids=None, resume=None, scale=None, out=None, workspace=None,
                       status=None, stream=None):
    """Linear attention over packed prompts: request b has tokens
    [cu_seqlens[b], cu_seqlens[b + 1]) of q [T, Hq, D] and k, v [T, Hkv, D]
    bf16, starts from its state where resume[b] != 0 (else from zero) and
    leaves its last state in the pool.  Returns out bf16 [T, Hq, D]; rows of
    no request are left as they were (unset in an output made here)."""
    dev = _device(q, torch.bfloat16, "q")
    B = _shape(cu_seqlens, torch.int32, dev, "cu_seqlens", 1)[0] - 1
    if B < 0:
        raise ValueError("cu_seqlens must be [batch + 1]")
    T, Hq, D, pc = _linear_args(q, k, v, pool, log_decay, state_ids, B, dev)
    if resume is not None and _shape(resume, torch.int32, dev, "resume", 1) != (B,):
        raise ValueError("resume must be [batch]")
    out = _linear_out(out, T, Hq, D, torch.bfloat16, dev, stream)
    if out.dtype != torch.bfloat16:
        raise ValueError("out must be bfloat16")
    ws, ws_bytes, _held = _call_memory(
        workspace, linear_prompt_workspace_bytes(B, Hq, pc.num_kv_heads, D, T, max_seq_len), dev,
        stream)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    _check(lib().phs_linear_attn_prompt(q.data_ptr(), Hq, k.data_ptr(), v.data_ptr(),
                                        cu_seqlens.data_ptr(), T, int(max_seq_len), pc,
                                        _ptr(state_ids), _ptr(resume), log_decay.data_ptr(), B,
                                        scale, out.data_ptr(), ws, ws_bytes,
                                        _status_ptr(status, dev), _raw_stream(stream, dev)),
           "linear_attn_prompt")
    return out


# ------------------------------------------- rotary positions, cache writes --
def _rows(t, dtype, dev, name, dims):
    """(shape, row stride) of t: rows of a token side by side in memory, at
    any stride (a part of a wider projection's output)."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev:
        shape = t.shape
        if len(shape) == dims:
            strides = t.stride()
            cols = shape[1] if dims == 2 else shape[1] * shape[2]
            if (strides[-1] == 1 or shape[-1] == 1) and \
                    (dims == 2 or strides[1] == shape[2] or shape[1] == 1):
                return shape, strides[0] if shape[0] > 1 else cols
            if cols == 0 or shape[0] == 0:
                return shape, cols
            raise ValueError(f"{name}: a token's elements must lie side by side")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype or t.dim() != dims or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor of {dims} dims and {dtype}")
    raise ValueError(_DEVICE_ERROR)


@dataclass
class Rope:
    """Rotary positions: turns int64 [rotary_dim / 2], the share of a full
    turn that each position adds to pair i's angle, as a 64-bit fraction
    (stored in the int64's bits); pairs of elements i and i + rotary_dim / 2,
    with `interleaved` 2 i and 2 i + 1; cos and sin are multiplied by
    `factor`.  `make` lays out the usual ones."""
    turns: torch.Tensor
    interleaved: bool = False
    factor: float = 1.0

    def c(self, dev):
        half, = _shape(self.turns, torch.int64, dev, "rope.turns", 1)
        return _lib.RopeC(self.turns.data_ptr(), 2 * half, self.interleaved, self.factor)

    @staticmethod
    def make(rotary_dim, base=10000.0, interleaved=False, scaling=None, scale=1.0,
             trained_len=None, low=None, high=None, factor=None, device="cuda"):
        """Pair i turns by base^(-2 i / rotary_dim) radians a position.
        Scalings to contexts `scale` times as long:
          "linear"       all pairs `scale` times slower;
          "base"         the base raised so that the slowest pair is `scale`
                         times slower and the fastest as it was;
          "parts"        pairs of more than `high` (32) rotations in trained_len
                         as they were, of fewer than `low` (1) `scale` times
                         slower, between them by their index; factor
                         0.1 ln(scale) + 1;
          "wavelengths"  the same with 4 and 1, between them by their
                         rotations.
        factor: the one of cos and sin, where it is not the scaling's."""
        freq, mag = rope_frequencies(rotary_dim, base, scaling, scale, trained_len, low, high)
        import numpy as np
        turns = np.array([round(f / (2 * math.pi) * 2.0 ** 64) % 2 ** 64 for f in freq.tolist()],
                         dtype=np.uint64)
        return Rope(torch.from_numpy(turns.view(np.int64)).to(device), interleaved,
                    float(mag if factor is None else factor))


def rope_frequencies(rotary_dim, base=10000.0, scaling=None, scale=1.0, trained_len=None, low=None,
                     high=None):
    """(radians a position of each pair, host fp64 [rotary_dim / 2]; factor of
    cos and sin) of Rope.make's scalings."""
    import numpy as np
    if rotary_dim <= 0 or rotary_dim % 2 or not base > 1 or not scale >= 1:
        raise ValueError("rotary_dim must be even and positive, base above 1, scale at least 1")
    half = rotary_dim // 2
    i = np.arange(half)
    if scaling == "base":
        if half < 2:
            raise ValueError("scaling of the base needs at least two pairs")
        base = base * scale ** (half / (half - 1))
    freq = float(base) ** (-i / half)
    if scaling in (None, "base"):
        return freq, 1.0
    if scaling == "linear":
        return freq / scale, 1.0
    if scaling not in ("parts", "wavelengths"):
        raise ValueError("scaling must be linear, base, parts or wavelengths")
    low = 1.0 if low is None else float(low)
    high = (32.0 if scaling == "parts" else 4.0) if high is None else float(high)
    if trained_len is None or trained_len <= 0 or not 0 < low < high:
        raise ValueError(f"scaling by {scaling} needs trained_len and 0 < low < high")
    if scaling == "parts":
        # index of the pair that makes so many rotations in trained_len
        at = [half * math.log(trained_len / (2 * math.pi * r)) / math.log(base)
              for r in (high, low)]
        # (`last` may lie behind the slowest pair, which then keeps a part of its speed)
        first, last = max(math.floor(at[0]), 0), math.ceil(at[1])
        slow = np.clip((i - first) / max(last - first, 0.001), 0, 1)
        return freq * (1 - slow) + freq / scale * slow, 0.1 * math.log(scale) + 1
    keep = np.clip((trained_len * freq / (2 * math.pi) - low) / (high - low), 0, 1)
    return freq * keep + freq / scale * (1 - keep), 1.0


def rope_rotate(q, k, positions, rope: Rope, q_out=None, k_out=None, stream=None):
    """q [T, Hq, D] and k [T, Hkv, D] (None: q alone) bf16, rotated by
    positions int32 [T] into q_out, k_out (may be the inputs themselves);
    returns (q_out, k_out).  For layers whose attention call appends k itself."""
    dev = _device(q, torch.bfloat16, "q")
    (T, Hq, D), qs = _rows(q, torch.bfloat16, dev, "q", 3)
    Hk = ks = kos = 0
    if k is not None:
        (Tk, Hk, Dk), ks = _rows(k, torch.bfloat16, dev, "k", 3)
        if Tk != T or Dk != D:
            raise ValueError("q and k differ in tokens or head_dim")
    if _shape(positions, torch.int32, dev, "positions", 1) != (T,):
        raise ValueError("positions must be [tokens]")
    if q_out is None:
        q_out = _empty((T, Hq, D), torch.bfloat16, dev, stream)
    shape, qos = _rows(q_out, torch.bfloat16, dev, "q_out", 3)
    if shape != (T, Hq, D):
        raise ValueError("q_out must have q's shape")
    if k is None:
        if k_out is not None:
            raise ValueError("k_out without k")
    else:
        if k_out is None:
            k_out = _empty((T, Hk, D), torch.bfloat16, dev, stream)
        shape, kos = _rows(k_out, torch.bfloat16, dev, "k_out", 3)
        if shape != (T, Hk, D):
            raise ValueError("k_out must have k's shape")
    _check(lib().phs_rope_rotate(q.data_ptr(), qs, Hq, _ptr(k), ks, Hk, D, T,
                                 positions.data_ptr(), rope.c(dev), q_out.data_ptr(), qos,
                                 _ptr(k_out), kos, _raw_stream(stream, dev)), "rope_rotate")
    return q_out, k_out


def _int8_c(int8, dev):
    n, h, q, d = _shape(int8.k, torch.uint8, dev, "int8.k", 4)
    if q != QBLOCK or \
            _shape(int8.v, torch.uint8, dev, "int8.v", 5) != (n, h, 2, d, QBLOCK // 2) or \
            _shape(int8.k_scale, torch.float32, dev, "int8.k_scale", 2) != (n, h) or \
            _shape(int8.v_scale, torch.float32, dev, "int8.v_scale", 2) != (n, h):
        raise ValueError("inconsistent INT8 pool shapes")
    return _lib.Int8PoolC(int8.k.data_ptr(), int8.v.data_ptr(), int8.k_scale.data_ptr(),
                          int8.v_scale.data_ptr(), n, h, d)


def _per_request(t, dev, name, batch):
    if _shape(t, torch.int32, dev, name, 1) != (batch,):
        raise ValueError(f"{name} needs one entry per request")
    return t.data_ptr()


def kv_write_paged(pool: PagedPool, k, v, block_table, seq_lens, cu_seqlens=None,
                   rope: Rope | None = None, q=None, q_out=None, int8: Int8Pool | None = None,
                   qtable=None, qlens_before=None, qlens=None, max_qblocks=0, page_refcount=None,
                   status=None, stream=None):
    """Write the new tokens of every request into the paged cache: k, v bf16
    [T, Hkv, D], request b's rows [cu_seqlens[b], cu_seqlens[b + 1]) (None: one
    token each), the last of its seq_lens[b] tokens.  With rope k is rotated by
    each token's place in its request, and q [T, Hq, D] into q_out, which is
    returned (None without q).  With int8 the blocks of 32 tokens from
    qlens_before[b] to qlens[b] (at most max_qblocks) are quantised, new tokens
    straight from k and v, earlier ones from their pages."""
    dev = _device(k, torch.bfloat16, "k")
    (T, H, D), ks = _rows(k, torch.bfloat16, dev, "k", 3)
    shape, vs = _rows(v, torch.bfloat16, dev, "v", 3)
    pc = _pool_c(pool, dev)
    if shape != (T, H, D) or H != pc.num_kv_heads or D != pc.head_dim:
        raise ValueError("k and v must be [tokens, Hkv of the pool, head_dim]")
    B, width = _shape(block_table, torch.int32, dev, "block_table", 2)
    lens = _per_request(seq_lens, dev, "seq_lens", B)
    cu = None
    if cu_seqlens is not None:
        cu = _per_request(cu_seqlens, dev, "cu_seqlens", B + 1)
    elif T != B:
        raise ValueError("without cu_seqlens one token per request")
    Hq = qs = 0
    if q is None:
        if q_out is not None:
            raise ValueError("q_out without q")
    else:
        if rope is None:
            raise ValueError("q goes with rope")
        (Tq, Hq, Dq), qs = _rows(q, torch.bfloat16, dev, "q", 3)
        if Tq != T or Dq != D:
            raise ValueError("q must be [tokens, Hq, head_dim]")
        if q_out is None:
            q_out = _empty((T, Hq, D), torch.bfloat16, dev, stream)
        elif _shape(q_out, torch.bfloat16, dev, "q_out", 3) != (T, Hq, D):
            raise ValueError("q_out must have q's shape")
    ic = qt = qb = ql = None
    qw = 0
    if int8 is not None:
        ic = _int8_c(int8, dev)
        rows, qw = _shape(qtable, torch.int32, dev, "qtable", 2)
        if rows != B:
            raise ValueError("qtable needs one row per request")
        qt = qtable.data_ptr()
        qb = _per_request(qlens_before, dev, "qlens_before", B)
        ql = _per_request(qlens, dev, "qlens", B)
    elif qtable is not None or qlens is not None or qlens_before is not None:
        raise ValueError("qtable and qlens go with int8")
    if page_refcount is not None and \
            _shape(page_refcount, torch.int32, dev, "page_refcount", 1) != (pc.num_pages,):
        raise ValueError("page_refcount needs one entry per page")
    _check(lib().phs_kv_write_paged(
        pc, k.data_ptr(), ks, v.data_ptr(), vs, T, cu, block_table.data_ptr(), width, lens, B,
        None if rope is None else rope.c(dev), _ptr(q), qs, Hq, _ptr(q_out), ic, qt, qw, qb, ql,
        int(max_qblocks), _ptr(page_refcount), _status_ptr(status, dev), _raw_stream(stream, dev)),
        "kv_write_paged")
    return q_out


def kv_read_paged(pool: PagedPool, block_table, starts, cu_seqlens, total_tokens: int,
                  max_tokens: int, int8: Int8Pool | None = None, qtable=None, qlens=None,
                  k_out=None, v_out=None, status=None, stream=None):
    """Tokens [starts[b], starts[b] + n) of every request, n = cu_seqlens[b + 1]
    - cu_seqlens[b] <= max_tokens, back from the cache as rows [cu_seqlens[b],
    ...) of bf16 [total_tokens, Hkv, D]; those below qlens[b] from their 8-bit
    blocks.  Returns (k_out, v_out)."""
    dev = _device(block_table, torch.int32, "block_table")
    B, width = _shape(block_table, torch.int32, dev, "block_table", 2)
    pc = _pool_c(pool, dev)
    at = _per_request(starts, dev, "starts", B)
    cu = _per_request(cu_seqlens, dev, "cu_seqlens", B + 1)
    shape = (int(total_tokens), pc.num_kv_heads, pc.head_dim)
    if k_out is None:
        k_out = _empty(shape, torch.bfloat16, dev, stream)
    if v_out is None:
        v_out = _empty(shape, torch.bfloat16, dev, stream)
    if _shape(k_out, torch.bfloat16, dev, "k_out", 3) != shape or \
            _shape(v_out, torch.bfloat16, dev, "v_out", 3) != shape:
        raise ValueError("k_out and v_out must be [total_tokens, Hkv, head_dim]")
    ic = qt = ql = None
    qw = 0
    if int8 is not None:
        ic = _int8_c(int8, dev)
        rows, qw = _shape(qtable, torch.int32, dev, "qtable", 2)
        if rows != B:
            raise ValueError("qtable needs one row per request")
        qt = qtable.data_ptr()
        ql = _per_request(qlens, dev, "qlens", B)
    elif qtable is not None or qlens is not None:
        raise ValueError("qtable and qlens go with int8")
    _check(lib().phs_kv_read_paged(pc, block_table.data_ptr(), width, at, cu, B, shape[0],
                                   int(max_tokens), ic, qt, qw, ql, k_out.data_ptr(),
                                   v_out.data_ptr(), _status_ptr(status, dev),
                                   _raw_stream(stream, dev)), "kv_read_paged")
    return k_out, v_out


# ------------------------------------------------------- causal convolution --
@dataclass
class ConvPool:
    """Last inputs of a causal convolution: c bf16 [num_states, width - 1,
    channels], oldest first."""
    c: torch.Tensor

    @staticmethod
    def zeros(num_states, channels, width, device="cuda"):
        return ConvPool(torch.zeros((num_states, width - 1, channels), dtype=torch.bfloat16,
                                    device=device))


@dataclass
class ConvWeights:
    """Filters of a causal convolution: weight fp32 [channels, width], bias
    fp32 [channels] or None; with silu the sum y goes out as y / (1 + exp(-y))."""
    weight: torch.Tensor
    bias: torch.Tensor | None = None
    silu: bool = True


def _conv_args(x, pool, weights, state_ids, batch, out, dev, stream):
    """(row stride, descriptors of pool and weights, pointer of the ids, out)"""
    (T, C), stride = _rows(x, torch.bfloat16, dev, "x", 2)
    n, w1, channels = _shape(pool.c, torch.bfloat16, dev, "pool.c", 3)
    if C != channels:
        raise ValueError("x must be [tokens, channels of the pool]")
    if _shape(weights.weight, torch.float32, dev, "weight", 2) != (C, w1 + 1):
        raise ValueError("weight must be [channels, width]")
    bias = weights.bias
    if bias is not None and _shape(bias, torch.float32, dev, "bias", 1) != (C,):
        raise ValueError("bias must be [channels]")
    ids = None if state_ids is None else _per_request(state_ids, dev, "state_ids", batch)
    if out is None:
        out = _empty((T, C), torch.bfloat16, dev, stream)
    elif _shape(out, torch.bfloat16, dev, "out", 2) != (T, C):
        raise ValueError("out must have x's shape")
    return (stride, _lib.ConvPoolC(pool.c.data_ptr(), n, C, w1 + 1),
            _lib.ConvWeightsC(weights.weight.data_ptr(), _ptr(bias), weights.silu), ids, out)


def causal_conv_decode(x, pool: ConvPool, weights: ConvWeights, state_ids=None, out=None,
                       status=None, stream=None):
    """One token per request: x [B, channels] bf16; returns out [B, channels]
    and moves the requests' last inputs on by one."""
    dev = _device(x, torch.bfloat16, "x")
    B = x.shape[0]
    stride, pc, wc, ids, out = _conv_args(x, pool, weights, state_ids, B, out, dev, stream)
    _check(lib().phs_causal_conv_decode(x.data_ptr(), stride, pc, wc, ids, B, out.data_ptr(),
                                        _status_ptr(status, dev), _raw_stream(stream, dev)),
           "causal_conv_decode")
    return out


def causal_conv_prompt(x, cu_seqlens, pool: ConvPool, weights: ConvWeights, state_ids=None,
                       resume=None, out=None, status=None, stream=None):
    """The convolution over packed prompts: request b has rows [cu_seqlens[b],
    cu_seqlens[b + 1]) of x [T, channels] bf16, behind its last inputs in the
    pool where resume[b] != 0 (else behind zeros), and leaves its own there.
    Returns out [T, channels]; rows of no request are left as they were (unset
    in an output made here)."""
    dev = _device(x, torch.bfloat16, "x")
    B = _shape(cu_seqlens, torch.int32, dev, "cu_seqlens", 1)[0] - 1
    if B < 0:
        raise ValueError("cu_seqlens must be [batch + 1]")
    stride, pc, wc, ids, out = _conv_args(x, pool, weights, state_ids, B, out, dev, stream)
    again = None if resume is None else _per_request(resume, dev, "resume", B)
    _check(lib().phs_causal_conv_prompt(x.data_ptr(), stride, cu_seqlens.data_ptr(), x.shape[0],
                                        pc, wc, ids, again, B, out.data_ptr(),
                                        _status_ptr(status, dev), _raw_stream(stream, dev)),
           "causal_conv_prompt")
    return out


# ----------------------------------------------------------- selective scan --
@dataclass
class ScanPool:
    """States of a selective scan: s fp32 [num_states, H, P, N]."""
    s: torch.Tensor

    @staticmethod
    def zeros(num_states, num_heads, head_dim, state_dim, device="cuda"):
        return ScanPool(torch.zeros((num_states, num_heads, head_dim, state_dim),
                                    dtype=torch.float32, device=device))


@dataclass
class ScanWeights:
    """Weights of a selective scan, fp32 [H] each: the rate (<= 0), and where
    there are any the skip of x past the scan and the bias of the steps."""
    rate: torch.Tensor
    skip: torch.Tensor | None = None
    dt_bias: torch.Tensor | None = None


def _scan_args(x, dt, b, c, pool, weights, dev):
    """(tokens, groups, descriptors of inputs, pool and weights)"""
    shape, xs = _rows(x, torch.bfloat16, dev, "x", 3)
    T, H, P = shape
    bshape, bs = _rows(b, torch.bfloat16, dev, "b", 3)
    cshape, cs = _rows(c, torch.bfloat16, dev, "c", 3)
    kind = torch.float32 if isinstance(dt, torch.Tensor) and dt.dtype is torch.float32 \
        else torch.bfloat16
    dshape, ds = _rows(dt, kind, dev, "dt", 2)
    n, Hs, Ps, N = _shape(pool.s, torch.float32, dev, "pool.s", 4)
    if (Hs, Ps) != (H, P):
        raise ValueError("x must be [tokens, H, P] of the pool")
    if bshape != cshape or bshape[0] != T or bshape[2] != N:
        raise ValueError("b and c must be [tokens, groups, N of the pool]")
    if dshape != (T, H):
        raise ValueError("dt must be [tokens, H]")
    rate = _shape(weights.rate, torch.float32, dev, "rate", 1)
    if rate != (H,):
        raise ValueError("rate must be [H]")
    skip, bias = weights.skip, weights.dt_bias
    if skip is not None and _shape(skip, torch.float32, dev, "skip", 1) != rate or \
            bias is not None and _shape(bias, torch.float32, dev, "dt_bias", 1) != rate:
        raise ValueError("skip and dt_bias must be [H]")
    return (T, bshape[1],
            _lib.ScanInputsC(x.data_ptr(), b.data_ptr(), c.data_ptr(), dt.data_ptr(), xs, bs, cs,
                             ds, bshape[1], OUT_F32 if kind is torch.float32 else OUT_BF16),
            _lib.ScanPoolC(pool.s.data_ptr(), n, H, P, N),
            _lib.ScanWeightsC(weights.rate.data_ptr(), _ptr(skip), _ptr(bias)))


def selective_scan_decode(x, dt, b, c, pool: ScanPool, weights: ScanWeights, state_ids=None,
                          out=None, out_dtype=torch.bfloat16, status=None, stream=None):
    """One token of a selective scan per request: x [B, H, P], b, c [B, G, N]
    bf16, dt [B, H] bf16 or fp32; updates the states and returns out
    [B, H, P]."""
    dev = _device(x, torch.bfloat16, "x")
    B, _, ic, pc, wc = _scan_args(x, dt, b, c, pool, weights, dev)
    ids = None if state_ids is None else _per_request(state_ids, dev, "state_ids", B)
    if out is None:
        out = _empty(x.shape, out_dtype, dev, stream)
    elif _shape(out, out.dtype, dev, "out", 3) != x.shape:
        raise ValueError("out must have x's shape")
    _check(lib().phs_selective_scan_decode(ic, pc, wc, ids, B, out.data_ptr(),
                                           _out_code(out.dtype), _status_ptr(status, dev),
                                           _raw_stream(stream, dev)), "selective_scan_decode")
    return out


def scan_prompt_workspace_bytes(batch, num_heads, num_groups, head_dim, state_dim, total_tokens,
                                max_seq_len) -> int:
    """Workspace bytes for selective_scan_prompt; 0 if unsupported.  For a call
    of these very sizes: one with fewer requests may need more."""
    return int(lib().phs_scan_prompt_workspace_bytes(batch, num_heads, num_groups, head_dim,
                                                     state_dim, total_tokens, max_seq_len))


def selective_scan_prompt(x, dt, b, c, cu_seqlens, max_seq_len: int, pool: ScanPool,
                          weights: ScanWeights, state_ids=None, resume=None, out=None,
                          workspace=None, status=None, stream=None):
    """A selective scan over packed prompts: request b has tokens
    [cu_seqlens[b], cu_seqlens[b + 1]) of x [T, H, P], b, c [T, G, N] bf16 and
    dt [T, H] bf16 or fp32, starts from its state where resume[b] != 0 (else
    from zero) and leaves its last state in the pool.  Returns out bf16
    [T, H, P]; rows of no request are left as they were (unset in an output
    made here)."""
    dev = _device(x, torch.bfloat16, "x")
    B = _shape(cu_seqlens, torch.int32, dev, "cu_seqlens", 1)[0] - 1
    if B < 0:
        raise ValueError("cu_seqlens must be [batch + 1]")
    T, G, ic, pc, wc = _scan_args(x, dt, b, c, pool, weights, dev)
    ids = None if state_ids is None else _per_request(state_ids, dev, "state_ids", B)
    again = None if resume is None else _per_request(resume, dev, "resume", B)
    if out is None:
        out = _empty(x.shape, torch.bfloat16, dev, stream)
    elif _shape(out, torch.bfloat16, dev, "out", 3) != x.shape:
        raise ValueError("out must have x's shape")
    ws, ws_bytes, _held = _call_memory(
        workspace, scan_prompt_workspace_bytes(B, pc.num_heads, G, pc.head_dim, pc.state_dim, T,
                                               max_seq_len), dev, stream)
    _check(lib().phs_selective_scan_prompt(ic, cu_seqlens.data_ptr(), T, int(max_seq_len), pc, wc,
                                           ids, again, B, out.data_ptr(), ws, ws_bytes,
                                           _status_ptr(status, dev), _raw_stream(stream, dev)),
           "selective_scan_prompt")
    return out
