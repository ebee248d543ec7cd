"""Pools whose byte and element offsets pass 32 bits: the same results as with
the same pages and states at low ids."""
import numpy as np
import pytest
import torch

import paged_hybrid_sliding_gb300 as phs
import synth
from gpu_util import dev

pytestmark = pytest.mark.gpu


def test_pages_and_diff_decode_past_4_gb():
    heads, D, pages = 8, 128, 150_000        # 32 KB a page: 4.9 GB of K, as much of V
    big = phs.PagedPool.empty(pages, heads, D)
    used = [149_990, 149_999, 131_073, 3]    # 61 tokens
    small = phs.PagedPool(synth.normal_bf16((8, heads, 16, D), 1, device="cuda"),
                          synth.normal_bf16((8, heads, 16, D), 2, device="cuda"))
    for i, p in enumerate(used):
        big.k[p], big.v[p] = small.k[i], small.v[i]
    counts = torch.zeros(pages, dtype=torch.int32, device="cuda")
    counts[used] = 1
    table = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    table[0] = dev(used)
    lens = dev([61, 0])
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    vec = torch.full((D,), 0.03, device="cuda")
    w = phs.DiffWeights(vec, vec, -vec, vec, 0.4)
    q = synth.normal_bf16((1, 2 * 8, D), 3, device="cuda")

    def decode(pool, t, row, **kw):
        return phs.attn_decode_diff_paged(q, pool, t[row:row + 1], lens[:1], 64, w,
                                          out_dtype=torch.float32, status=st, **kw)

    want = decode(small, dev([[0, 1, 2, 3]]), 0)
    assert torch.equal(decode(big, table, 0), want)
    # a fork whose last page is copied from a high page to the lowest free one
    table[0] = dev([3, 131_073, 149_990, 149_999])
    low = dev([[3, 2, 0, 1]])
    want = decode(small, low, 0)
    phs.pages_fork([big], table, lens, counts, dev([0]), dev([1]), status=st)
    assert table[1].tolist() == [3, 131_073, 149_990, 0]
    assert torch.equal(big.k[0], small.k[1]) and torch.equal(big.v[0], small.v[1])
    assert torch.equal(decode(big, table, 1), want)
    # and everything down to the lowest ids
    page_map, live = phs.pages_compact([big], table, lens, counts, status=st)
    assert int(live.item()) == 5 and int(table.max()) == 4
    assert page_map[[0, 3, 149_999, 149_990, 131_073]].tolist() == [0, 3, 1, 2, 4]
    for row in (0, 1):
        assert torch.equal(decode(big, table, row), want)
    # the append too
    k1 = synth.normal_bf16((1, heads, D), 4, device="cuda")
    big2 = phs.PagedPool(big.k, big.v)
    high = dev([[149_998, 149_997, 149_996, 149_995]])
    for i, p in enumerate(high[0].tolist()):
        big2.k[p], big2.v[p] = small.k[i], small.v[i]
    assert torch.equal(decode(big2, high, 0, k_new=k1, v_new=k1),
                       decode(small, dev([[0, 1, 2, 3]]), 0, k_new=k1, v_new=k1))
    assert torch.equal(big2.k[149_995], small.k[3])
    assert int(st.item()) == 0


def test_states_past_31_bits():
    n, H, D, T = 4200, 32, 128, 200           # 2.2e9 elements, 8.8 GB
    big = phs.StatePool(torch.empty((n, H, D, D), device="cuda"))
    assert big.s.numel() > 2**31
    start = torch.randn((2, H, D, D), generator=torch.Generator(device="cuda").manual_seed(5),
                        device="cuda")
    ids = [4190, 4199]
    for i, x in zip(ids, start):
        big.s[i] = x
    small = phs.StatePool(start.clone())
    g = -torch.logspace(-3, -0.3, H, device="cuda")
    q, k, v = (synth.normal_bf16((2 * T, H, D), s, device="cuda") for s in (6, 7, 8))
    cu, res = dev([0, T, 2 * T]), dev([1, 1])
    a = phs.linear_attn_prompt(q, k, v, cu, T, big, g, state_ids=dev(ids), resume=res)
    b = phs.linear_attn_prompt(q, k, v, cu, T, small, g, resume=res)
    assert torch.equal(a, b)
    a = phs.linear_attn_decode(q[:2], k[:2], v[:2], big, g, state_ids=dev(ids))
    b = phs.linear_attn_decode(q[:2], k[:2], v[:2], small, g)
    assert torch.equal(a, b)
    assert torch.equal(big.s[ids], small.s)


def test_many_short_requests():
    """More requests than a warp, a tile or a CTA's threads hold."""
    B, H, D = 1500, 2, 64
    lens = np.random.RandomState(3).randint(0, 40, B)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T = int(cu[-1])
    q, k, v = (synth.normal_bf16((T, H, D), s, device="cuda") for s in (9, 10, 11))
    g = -torch.logspace(-2, -0.5, H, device="cuda")
    pool = phs.StatePool.zeros(B, H, D)
    out = phs.linear_attn_prompt(q, k, v, dev(cu), 40, pool, g)
    for b in (0, 31, 32, 639, 640, 1023, 1024, 1499):
        a, e = int(cu[b]), int(cu[b + 1])
        one = phs.StatePool.zeros(1, H, D)
        ref = phs.linear_attn_prompt(q[a:e], k[a:e], v[a:e], dev([0, e - a]), 40, one, g)
        assert torch.equal(out[a:e], ref), b
        assert torch.equal(pool.s[b], one.s[0]), b
