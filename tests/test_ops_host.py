"""Refusals and host bookkeeping of the page operations, differential
attention and linear attention that need no GPU: every call here is refused
before anything is launched."""
import ctypes

import numpy as np
import pytest
import torch

import ops_ref
import paged_hybrid_sliding_gb300 as phs
from paged_hybrid_sliding_gb300 import _lib

P = ctypes.c_void_p(1 << 20)   # an aligned address that no refused call reads
ODD = ctypes.c_void_p((1 << 20) + 8)


def paged(**kw):
    f = dict(k=P.value, v=P.value, num_pages=8, page_size=16, num_kv_heads=4, head_dim=64) | kw
    return _lib.PagedPoolC(*f.values())


def ref(x):
    return ctypes.byref(x)


@pytest.mark.parametrize("change,code", [
    (dict(table=None), -1), (dict(lens=None), -1), (dict(counts=None), -1), (dict(pages=0), -1),
    (dict(rows=None), -1), (dict(n=-1), -1), (dict(num_rows=0), -1), (dict(width=0), -1),
    (dict(width=1 << 28), -7), (dict(n=0), 0)])
def test_pages_free(change, code):
    a = dict(table=P, num_rows=4, width=4, lens=P, counts=P, pages=8, rows=P, n=2) | change
    assert phs.lib().phs_pages_free(*a.values(), None, None) == code


@pytest.mark.parametrize("change,code", [
    (dict(layers=0), -1), (dict(src=None), -1), (dict(n=-1), -1), (dict(ws=None), -5),
    (dict(size=8), -5), (dict(ws=ODD), -9), (dict(counts=None), -1), (dict(n=0), 0)])
def test_pages_fork(change, code):
    pools = (_lib.PagedPoolC * 2)(paged(), paged())
    a = dict(pools=pools, layers=2, table=P, num_rows=4, width=4, lens=P, counts=P, src=P, dst=P,
             n=2, ws=P, size=1 << 20) | change
    assert phs.lib().phs_pages_fork(*a.values(), None, None) == code


@pytest.mark.parametrize("pool,code", [
    (dict(num_kv_heads=2), -2), (dict(num_pages=9), -2), (dict(head_dim=128), -2),
    (dict(head_dim=96), -7), (dict(page_size=32), -7), (dict(k=ODD.value), -9),
    (dict(v=0), -1)])
def test_pages_compact_pools_must_be_alike(pool, code):
    pools = (_lib.PagedPoolC * 2)(paged(), paged(**pool))
    assert phs.lib().phs_pages_compact(pools, 2, P, 4, 4, P, P, P, P, P, P, P, 1 << 20, None,
                                       None) == code


def test_workspace_sizes():
    assert phs.pages_fork_workspace_bytes(0, 1) == 0
    assert phs.pages_fork_workspace_bytes(5, 3) > 0
    assert phs.pages_compact_workspace_bytes(0) == 0
    assert phs.pages_compact_workspace_bytes(1 << 31) == 0
    assert phs.pages_compact_workspace_bytes(1000) >= 12000
    assert phs.linear_prompt_workspace_bytes(1, 3, 2, 64, 10, 10) == 0
    assert phs.linear_prompt_workspace_bytes(1, 2, 2, 96, 10, 10) == 0
    assert phs.linear_prompt_workspace_bytes(-1, 2, 2, 64, 10, 10) == 0


@pytest.mark.parametrize("change,code", [
    (dict(q=None), -1), (dict(w=None), -1), (dict(scale=0.0), -1), (dict(scale=float("nan")), -1),
    (dict(dtype=2), -1), (dict(k_new=P), -1), (dict(k_new=ODD, v_new=P), -9),
    (dict(pool=paged(num_kv_heads=3)), -2), (dict(width=0), -1), (dict(out=None), -1)])
def test_diff(change, code):
    w = _lib.DiffWeightsC(P.value, P.value, P.value, P.value, 0, 0.5, 1e-5, 0)
    a = dict(q=P, heads=4, pool=paged(), table=P, width=4, lens=P, most=64, batch=2, w=w,
             scale=0.1, tps=0, out=P, dtype=1, ws=P, size=1 << 20, k_new=None,
             v_new=None) | change
    a["pool"] = ref(a["pool"])
    a["w"] = None if a["w"] is None else ref(a["w"])
    assert phs.lib().phs_attn_decode_diff_paged(*a.values(), None, None, None) == code


@pytest.mark.parametrize("bad", [dict(lambda_q1=0), dict(lambda_k2=0),
                                 dict(lambda_init=float("inf")), dict(norm_eps=-1.0),
                                 dict(norm_eps=float("nan"))])
def test_diff_weights(bad):
    f = dict(lambda_q1=P.value, lambda_k1=P.value, lambda_q2=P.value, lambda_k2=P.value,
             norm_weight=0, lambda_init=0.5, norm_eps=1e-5, lambda_per_head=0) | bad
    assert phs.lib().phs_attn_decode_diff_paged(
        P, 4, ref(paged()), P, 4, P, 64, 2, ref(_lib.DiffWeightsC(*f.values())), 0.1, 0, P, 1, P,
        1 << 20, None, None, None, None, None) == -1


@pytest.mark.parametrize("change,code", [
    (dict(pool=dict(s=0)), -1), (dict(pool=dict(n=0)), -1), (dict(pool=dict(d=96)), -7),
    (dict(heads=3), -2), (dict(heads=34), -7), (dict(q=None), -1), (dict(q=ODD), -9),
    (dict(decay=None), -1), (dict(batch=-1), -1), (dict(batch=9), -2),
    (dict(scale=float("nan")), -1), (dict(batch=0), 0)])
def test_linear(change, code):
    a = dict(q=P, heads=4, pool={}, k=P, v=P, decay=P, ids=None, batch=2, scale=0.1, out=P) | change
    s = dict(s=P.value, n=4, h=2, d=64) | a.pop("pool")
    pool = _lib.StatePoolC(*s.values())
    lib = phs.lib()
    assert lib.phs_linear_attn_decode(a["q"], a["heads"], ref(pool), a["k"], a["v"], a["decay"],
                                      a["ids"], a["batch"], a["scale"], a["out"], 0, None,
                                      None) == code
    assert lib.phs_linear_attn_prompt(a["q"], a["heads"], a["k"], a["v"], P, 100, 64, ref(pool),
                                      a["ids"], None, a["decay"], a["batch"], a["scale"], a["out"],
                                      P, 1 << 26, None, None) == code


@pytest.mark.parametrize("change,code", [
    (dict(cu=None), -1), (dict(tokens=-1), -1), (dict(most=-1), -1), (dict(ws=None), -5),
    (dict(ws=ODD), -9)])
def test_linear_prompt(change, code):
    a = dict(cu=P, tokens=100, most=64, ws=P) | change
    pool = _lib.StatePoolC(P.value, 4, 2, 64)
    assert phs.lib().phs_linear_attn_prompt(P, 4, P, P, a["cu"], a["tokens"], a["most"], ref(pool),
                                            None, None, P, 2, 0.1, P, a["ws"], 1 << 26, None,
                                            None) == code


def test_binding_wants_cuda_tensors():
    t = torch.zeros((2, 4), dtype=torch.int32)
    with pytest.raises(ValueError):
        phs.pages_free(t, t[0], t[0], t[0])
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        phs.linear_attn_decode(q, q, q, phs.StatePool.zeros(2, 4, 64, device="cpu"), torch.zeros(4))


# ------------------------------------------------- counts and ids come home --
def test_load_refcounts():
    a = phs.PageAllocator(6)
    a.load_refcounts([2, 0, 1, 0, 0, 7])
    assert a.refcounts().tolist() == [2, 0, 1, 0, 0, 7] and a.free_count() == 3
    assert a.alloc(2).tolist() == [1, 3]
    with pytest.raises(phs.PhsError):
        a.load_refcounts([1, 1, 1, -1, 1, 1])
    with pytest.raises(ValueError):
        a.load_refcounts([1, 1])
    assert a.refcounts().tolist() == [2, 1, 1, 1, 0, 7]


def test_radix_tree_follows_a_compaction():
    alloc = phs.PageAllocator(32)
    tree = phs.RadixTree(alloc, 16)
    gap = alloc.alloc(5)
    first = alloc.alloc(4)
    tokens = list(range(64)), list(range(32)) + list(range(900, 932))
    tree.insert(tokens[0], first)
    second = np.concatenate([first[:2], alloc.alloc(2)])
    tree.insert(tokens[1], second)
    alloc.decref(first)
    alloc.decref(second[2:])
    alloc.decref(gap)
    counts = alloc.refcounts()
    page_map, live = ops_ref.compact([], np.zeros((0, 1), np.int32), [], counts)
    alloc.load_refcounts(counts)
    tree.remap(page_map)
    assert live == 6
    for t, p in zip(tokens, (first, second)):
        hit = tree.match(t)
        assert hit.tolist() == page_map[p].tolist() and hit.max() < live
        alloc.decref(hit)
    # a map without a new id for a cached page is refused
    with pytest.raises(phs.PhsError) as e:
        tree.remap(np.full(32, -1, np.int32))
    assert e.value.code == -3
    with pytest.raises(phs.PhsError) as e:
        tree.remap(page_map[:9])
    assert e.value.code == -2
    assert tree.match(tokens[0]).tolist() == page_map[first].tolist()
