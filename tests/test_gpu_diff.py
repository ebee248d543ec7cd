"""Differential attention decode against the 64-bit definition."""
import math

import numpy as np
import pytest
import torch

import ops_ref
import paged_hybrid_sliding_gb300 as phs
import synth
from gpu_util import dev

pytestmark = pytest.mark.gpu


def make(lens, H, Hv, D, seed, per_head=False, norm=True, spare=3):
    lens = np.asarray(lens, np.int32)
    bt, npg = synth.block_tables_from_permutation(synth.pages_needed(np.maximum(lens, 1)), seed)
    npg += spare
    pool = phs.PagedPool(synth.normal_bf16((npg, 2 * Hv, 16, D), seed + 1, device="cuda"),
                         synth.normal_bf16((npg, 2 * Hv, 16, D), seed + 2, device="cuda"))
    q = synth.normal_bf16((len(lens), 2 * H, D), seed + 3, device="cuda") * 1.5
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (H, D) if per_head else (D,)
    lam = [torch.randn(shape, generator=g, device="cuda") * 0.2 for _ in range(4)]
    nw = 1 + 0.3 * torch.randn(2 * D, generator=g, device="cuda") if norm else None
    w = phs.DiffWeights(*lam, lambda_init=0.6, norm_weight=nw, norm_eps=1e-5)
    return pool, q, bt, lens, w


def check(out, pool, q, bt, lens, w, scale=None, hide=()):
    D = q.shape[2]
    ref, bound = ops_ref.diff_decode(
        q, pool.k, pool.v, bt, lens, (w.lambda_q1, w.lambda_k1, w.lambda_q2, w.lambda_k2),
        w.lambda_init, w.norm_weight, w.norm_eps, scale or 1 / math.sqrt(D),
        torch.finfo(out.dtype).eps / 2)
    err = (out.double() - ref).abs()
    assert torch.isfinite(out).all()
    worst = (err - bound).max()
    assert bool((err <= bound).all()), f"worst excess {float(worst):.3e}, err {float(err.max()):.3e}"


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("H,Hv", [(1, 1), (2, 2), (6, 2), (8, 1), (12, 1), (16, 1), (32, 4)])
def test_decode(D, dtype, H, Hv):
    pool, q, bt, lens, w = make([0, 1, 15, 16, 17, 130, 1000], H, Hv, D, 31 * H + D,
                                per_head=H == 6, norm=H != 8)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = phs.attn_decode_diff_paged(q, pool, dev(bt), dev(lens), 1000, w, out_dtype=dtype,
                                     status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert not out[0].any()
    check(out, pool, q, bt, lens, w)


@pytest.mark.parametrize("tps", [32, 128, 256, 4096])
def test_split_lengths(tps):
    pool, q, bt, lens, w = make([3000, 31, 32, 33, 257], 4, 2, 128, 5)
    out = phs.attn_decode_diff_paged(q, pool, dev(bt), dev(lens), 3000, w, out_dtype=torch.float32,
                                     tokens_per_split=tps)
    check(out, pool, q, bt, lens, w)


def test_long_cache():
    pool, q, bt, lens, w = make([40001, 7], 4, 1, 64, 6)
    out = phs.attn_decode_diff_paged(q, pool, dev(bt), dev(lens), 40001, w,
                                     out_dtype=torch.float32)
    check(out, pool, q, bt, lens, w)


def test_peaked_maps_and_scale():
    # one key far above the others in each map, at a different place
    pool, q, bt, lens, w = make([500, 77], 2, 1, 64, 7, norm=False)
    for b in range(2):
        for m, t in ((0, 3), (1, 70)):
            pool.k[int(bt[b, t // 16]), m, t % 16] = q[b, m] * 4
    out = phs.attn_decode_diff_paged(q, pool, dev(bt), dev(lens), 500, w, softmax_scale=0.5,
                                     out_dtype=torch.float32)
    check(out, pool, q, bt, lens, w, scale=0.5)


def test_equal_maps_with_lambda_one_cancel():
    """Both maps alike and lambda = 1: the difference is zero, and its norm
    is a division by the square root of eps, not by zero."""
    pool, q, bt, lens, w = make([100], 2, 1, 64, 8)
    pool.k[:, 1] = pool.k[:, 0]
    q[:, 1::2] = q[:, 0::2]
    z = torch.zeros(64, device="cuda")
    w = phs.DiffWeights(z, z, z, z, lambda_init=1.0, norm_weight=w.norm_weight)
    out = phs.attn_decode_diff_paged(q, pool, dev(bt), dev(lens), 100, w, out_dtype=torch.float32)
    assert torch.isfinite(out).all() and float(out.abs().max()) == 0.0


def test_infinities_and_nan_behind_the_last_token():
    pool, q, bt, lens, w = make([1, 17, 100, 250], 4, 2, 128, 9)
    for b, n in enumerate(lens):
        page, at = int(bt[b, (n - 1) // 16]), (n - 1) % 16 + 1
        pool.k[page, :, at:] = float("nan")
        pool.v[page, :, at:] = float("inf")
    out = phs.attn_decode_diff_paged(q, pool, dev(bt), dev(lens), 250, w, out_dtype=torch.float32)
    clean = phs.PagedPool(pool.k.nan_to_num(0, 0, 0), pool.v.nan_to_num(0, 0, 0))
    check(out, clean, q, bt, lens, w)


@pytest.mark.parametrize("D", [64, 128])
def test_fused_append_equals_append_then_decode(D):
    lens = [1, 16, 17, 300, 2049]
    pool, q, bt, lens, w = make(lens, 4, 2, D, 10)
    kn = synth.normal_bf16((5, 4, D), 77, device="cuda")
    vn = synth.normal_bf16((5, 4, D), 78, device="cuda")
    rc = torch.ones(pool.k.shape[0], dtype=torch.int32, device="cuda")
    rc[int(bt[3, 299 // 16])] = 2      # a shared page: not written
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    sep = phs.PagedPool(pool.k.clone(), pool.v.clone())
    out = phs.attn_decode_diff_paged(q, pool, dev(bt), dev(lens), 2049, w, k_new=kn, v_new=vn,
                                     page_refcount=rc, out_dtype=torch.float32, status=st)
    assert int(st.item()) == -4
    phs.kv_append_paged(sep, kn, vn, dev(bt), dev(lens), page_refcount=rc)
    ref = phs.attn_decode_diff_paged(q, sep, dev(bt), dev(lens), 2049, w, out_dtype=torch.float32)
    assert torch.equal(pool.k, sep.k) and torch.equal(pool.v, sep.v)
    assert torch.equal(out, ref)
    check(out, pool, q, bt, lens, w)


def test_bad_pages_and_lengths_are_recorded():
    pool, q, bt, lens, w = make([40, 40, 40], 4, 2, 64, 11)
    bt2 = bt.copy()
    bt2[1, 1] = 4000
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = phs.attn_decode_diff_paged(q, pool, dev(bt2), dev(lens), 40, w, status=st)
    assert int(st.item()) == -3
    good = phs.attn_decode_diff_paged(q, pool, dev(bt), dev(lens), 40, w)
    assert torch.equal(out[[0, 2]], good[[0, 2]])
    st.zero_()
    phs.attn_decode_diff_paged(q, pool, dev(bt), dev([40, 999, 40]), 48, w, status=st)
    assert int(st.item()) == -3
    st.zero_()
    out = phs.attn_decode_diff_paged(q, pool, dev(bt), dev([40, -1, 40]), 48, w, status=st)
    assert int(st.item()) == -3 and not out[1].any()


def test_side_stream_and_graph():
    pool, q, bt, lens, w = make([700, 33], 8, 2, 128, 12)
    bt_d, sl = dev(bt), dev(lens)
    out = torch.empty((2, 8, 256), dtype=torch.float32, device="cuda")
    ws = torch.empty(phs.diff_workspace_bytes(2, 8, 2, 128, 700), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    phs.attn_decode_diff_paged(q, pool, bt_d, sl, 700, w, out=out, workspace=ws, stream=s)
    s.synchronize()
    first = out.clone()
    check(first, pool, q, bt, lens, w)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        phs.attn_decode_diff_paged(q, pool, bt_d, sl, 700, w, out=out, workspace=ws)
    sl.copy_(dev([650, 20]))
    for _ in range(2):
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        check(out, pool, q, bt, np.array([650, 20]), w)


def test_what_follows_a_call_of_one_split_waits_for_it():
    """Where no request is split the second launch has nothing to do, and must
    not let the next work of a stream or graph start before the first is done."""
    pool, q, bt, lens, w = make([4000, 3500, 3999], 4, 2, 128, 9)
    args = (q, pool, dev(bt), dev(lens), 4096, w)
    kw = dict(out_dtype=torch.float32, tokens_per_split=4096)
    want = phs.attn_decode_diff_paged(*args, **kw)
    need = phs.diff_workspace_bytes(3, 4, 2, 128, 4096, 4096)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    out, copy = torch.empty_like(want), torch.empty_like(want)

    def step():
        out.zero_()
        phs.attn_decode_diff_paged(*args, out=out, workspace=ws, **kw)
        copy.copy_(out)

    step()
    torch.cuda.synchronize()
    assert torch.equal(copy, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(5):
        copy.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(copy, want)


def test_refusals():
    pool, q, bt, lens, w = make([40], 4, 2, 64, 13)
    a = (dev(bt), dev(lens), 40)

    def code(c, **kw):
        with pytest.raises(phs.PhsError) as e:
            phs.attn_decode_diff_paged(kw.pop("q", q), kw.pop("pool", pool), *a, kw.pop("w", w), **kw)
        assert e.value.code == c

    code(-1, softmax_scale=0.0)
    code(-1, softmax_scale=float("nan"))
    code(-5, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    code(-7, tokens_per_split=48)
    code(-2, q=synth.normal_bf16((1, 6, 64), 1, device="cuda"))      # 3 heads on 2 value heads
    code(-7, q=synth.normal_bf16((1, 68, 64), 1, device="cuda"))     # 17 heads a value head
    code(-1, w=phs.DiffWeights(w.lambda_q1, w.lambda_k1, w.lambda_q2, w.lambda_k2, float("nan")))
    with pytest.raises(ValueError):   # odd number of query rows
        phs.attn_decode_diff_paged(q[:, :7].contiguous(), pool, *a, w)
    with pytest.raises(ValueError):   # odd number of pool heads
        phs.attn_decode_diff_paged(q, phs.PagedPool.empty(4, 3, 64), *a, w)
    with pytest.raises(ValueError):   # lambda of another width
        phs.attn_decode_diff_paged(q, pool, *a, phs.DiffWeights(
            *[torch.zeros(32, device="cuda")] * 4, lambda_init=0.1))
    with pytest.raises(ValueError):   # norm of one map's width
        phs.attn_decode_diff_paged(q, pool, *a, phs.DiffWeights(
            *[torch.zeros(64, device="cuda")] * 4, lambda_init=0.1,
            norm_weight=torch.zeros(64, device="cuda")))
    with pytest.raises(ValueError):   # k_new without v_new
        phs.attn_decode_diff_paged(q, pool, *a, w, k_new=q[:, :4].contiguous())
