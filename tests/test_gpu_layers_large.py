"""Pools and rows whose offsets pass 32 bits, many short requests: the same
results as with the same pages, states and rows at low addresses."""
import numpy as np
import pytest
import torch

import paged_hybrid_sliding_gb300 as phs
import synth
from gpu_util import dev

pytestmark = pytest.mark.gpu


def test_cache_past_4_gb():
    heads, D, pages, qpages = 8, 128, 150_000, 70_000   # 4.9 GB of K; 2.3 GB of its codes
    n = 100
    k, v, q = (synth.normal_bf16((n, h, D), s, device="cuda") for h, s in ((8, 1), (8, 2), (16, 3)))
    rope = phs.Rope.make(128)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def write(pool, int8, table, qtable):
        qo = phs.kv_write_paged(pool, k, v, dev([table]), dev([n]), cu_seqlens=dev([0, n]), q=q,
                                rope=rope, int8=int8, qtable=dev([qtable]), qlens_before=dev([0]),
                                qlens=dev([64]), max_qblocks=2, status=st)
        return qo, *phs.kv_read_paged(pool, dev([table]), dev([0]), dev([0, n]), n, n, int8=int8,
                                      qtable=dev([qtable]), qlens=dev([64]), status=st)

    small = write(phs.PagedPool.empty(8, heads, D), phs.Int8Pool.empty(2, heads, D),
                  [0, 1, 2, 3, 4, 5, 6], [1, 0])
    big = write(phs.PagedPool.empty(pages, heads, D), phs.Int8Pool.empty(qpages, heads, D),
                [0, 1, 2, 3, 149_999, 131_073, 149_990], [69_999, 66_000])
    assert int(st.item()) == 0
    for a, b in zip(small, big):
        assert torch.equal(a, b)


def test_states_past_31_bits():
    n, H, P, N, T = 2200, 64, 128, 128, 200               # 2.3e9 elements, 9.2 GB
    big = phs.ScanPool(torch.empty((n, H, P, N), device="cuda"))
    assert big.s.numel() > 2**31
    start = torch.randn((2, H, P, N), generator=torch.Generator(device="cuda").manual_seed(5),
                        device="cuda")
    ids = [2190, 2199]
    for i, x in zip(ids, start):
        big.s[i] = x
    small = phs.ScanPool(start.clone())
    w = phs.ScanWeights(-torch.logspace(-3, 0.5, H, device="cuda"))
    x = synth.normal_bf16((2 * T, H, P), 6, device="cuda")
    b, c = (synth.normal_bf16((2 * T, 2, N), s, device="cuda") for s in (7, 8))
    dt = synth.normal_bf16((2 * T, H), 9, device="cuda")
    cu, res = dev([0, T, 2 * T]), dev([1, 1])
    one = phs.selective_scan_prompt(x, dt, b, c, cu, T, big, w, state_ids=dev(ids), resume=res)
    two = phs.selective_scan_prompt(x, dt, b, c, cu, T, small, w, resume=res)
    assert torch.equal(one, two)
    one = phs.selective_scan_decode(x[:2], dt[:2], b[:2], c[:2], big, w, state_ids=dev(ids))
    two = phs.selective_scan_decode(x[:2], dt[:2], b[:2], c[:2], small, w)
    assert torch.equal(one, two)
    assert torch.equal(big.s[ids], small.s)


def test_rows_past_31_bits():
    """Rows of a very wide projection: the last ones begin past 2^31 elements."""
    T, wide = 3000, 800_000                               # 2.4e9 elements, 4.8 GB
    C, H, P, N = 256, 2, 64, 64                           # x, b and c of the scan: 256 columns
    rows = torch.empty((T, wide), dtype=torch.bfloat16, device="cuda")
    x = synth.normal_bf16((T, C), 1, device="cuda")
    rows[:, 8:8 + C] = x
    far = rows[:, 8:8 + C]
    assert far.stride(0) * (T - 1) > 2**31
    w = phs.ConvWeights(torch.randn(C, 4, device="cuda"))
    cu = dev([0, 1100, T])
    outs = [phs.causal_conv_prompt(t, cu, phs.ConvPool.zeros(2, C, 4), w) for t in (x, far)]
    assert torch.equal(*outs)
    dt = synth.normal_bf16((T, H), 2, device="cuda")
    w = phs.ScanWeights(torch.tensor([-0.1, -1.0], device="cuda"))
    outs = []
    for t in (x, far):
        a = (t[:, :128].unflatten(1, (H, P)), dt, t[:, 128:192].unflatten(1, (1, N)),
             t[:, 192:].unflatten(1, (1, N)))
        pool = phs.ScanPool.zeros(2, H, P, N)
        outs.append((phs.selective_scan_prompt(*a, cu, T, pool, w), pool.s))
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    rope = phs.Rope.make(64)
    outs = [phs.rope_rotate(t.unflatten(1, (4, 64)), t[:, :64].unflatten(1, (1, 64)), pos, rope)
            for t in (x, far)]
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    table = dev(np.arange(T // 16 + 1)[None])
    pools = []
    for t in (x, far):
        pools.append(phs.PagedPool(*(torch.zeros((T // 16 + 1, 2, 16, 64), dtype=torch.bfloat16,
                                                 device="cuda") for _ in range(2))))
        phs.kv_write_paged(pools[-1], t[:, :128].unflatten(1, (2, 64)),
                           t[:, 128:].unflatten(1, (2, 64)), table, dev([T]), cu_seqlens=dev([0, T]))
    assert torch.equal(pools[0].k, pools[1].k) and torch.equal(pools[0].v, pools[1].v)


def test_many_short_requests():
    """More requests than a warp, a tile or a CTA's threads hold."""
    B, H, P, N, C = 1500, 2, 64, 64, 64
    lens = np.random.RandomState(3).randint(0, 40, B)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T = int(cu[-1])
    x, dt = synth.normal_bf16((T, H, P), 1, device="cuda"), synth.normal_bf16((T, H), 2, device="cuda")
    b, c = (synth.normal_bf16((T, 1, N), s, device="cuda") for s in (3, 4))
    ws = phs.ScanWeights(torch.tensor([-0.1, -1.0], device="cuda"))
    wc = phs.ConvWeights(torch.randn(C, 4, device="cuda"))
    scans, convs = phs.ScanPool.zeros(B, H, P, N), phs.ConvPool.zeros(B, C, 4)
    rows = x[:, 0]
    out = phs.selective_scan_prompt(x, dt, b, c, dev(cu), 40, scans, ws)
    conv = phs.causal_conv_prompt(rows, dev(cu), convs, wc)
    k = x
    table = dev(np.arange(3 * B).reshape(B, 3))
    pool = phs.PagedPool(*(torch.zeros((3 * B, H, 16, P), dtype=torch.bfloat16, device="cuda")
                           for _ in range(2)))
    phs.kv_write_paged(pool, k, k, table, dev(lens), cu_seqlens=dev(cu), rope=phs.Rope.make(64))
    ko, vo = phs.kv_read_paged(pool, table, dev(np.zeros(B)), dev(cu), T, 40)
    pos = torch.cat([torch.arange(int(n)) for n in lens]).int().cuda()
    assert torch.equal(vo, k)
    assert torch.equal(ko, phs.rope_rotate(k, None, pos, phs.Rope.make(64))[0])
    for r in (0, 31, 32, 639, 640, 1023, 1024, 1499):
        a, e = int(cu[r]), int(cu[r + 1])
        one = phs.ScanPool.zeros(1, H, P, N)
        want = phs.selective_scan_prompt(x[a:e], dt[a:e], b[a:e], c[a:e], dev([0, e - a]), 40, one,
                                         ws)
        assert torch.equal(out[a:e], want), r
        assert torch.equal(scans.s[r], one.s[0]), r
        one = phs.ConvPool.zeros(1, C, 4)
        want = phs.causal_conv_prompt(rows[a:e], dev([0, e - a]), one, wc)
        assert torch.equal(conv[a:e], want) and torch.equal(convs.c[r], one.c[0]), r


def test_nothing_to_do():
    """No tokens, no requests: states that are not continued become zero."""
    pool = phs.ScanPool(torch.ones((3, 2, 64, 64), device="cuda"))
    w = phs.ScanWeights(torch.tensor([-0.1, -1.0], device="cuda"))
    none = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")
    a = (none(0, 2, 64), none(0, 2), none(0, 1, 64), none(0, 1, 64))
    out = phs.selective_scan_prompt(*a, dev([0, 0, 0]), 0, pool, w, resume=dev([1, 0]))
    assert out.shape == (0, 2, 64)
    assert bool((pool.s[[0, 2]] == 1).all()) and not pool.s[1].any()
    phs.selective_scan_prompt(*a, dev([0]), 0, pool, w)
    assert phs.selective_scan_decode(*a, pool, w).shape == (0, 2, 64)
    kv = phs.PagedPool.empty(2, 2, 64)
    assert phs.kv_write_paged(kv, none(0, 2, 64), none(0, 2, 64), dev(np.zeros((0, 1))), dev([])) is None
    k, v = phs.kv_read_paged(kv, dev([[0]]), dev([0]), dev([0, 0]), 0, 0)
    assert k.shape == v.shape == (0, 2, 64)
    assert phs.rope_rotate(none(0, 2, 64), None, dev([]), phs.Rope.make(64))[0].shape == (0, 2, 64)


def test_old_tokens_into_8_bits_without_new_ones():
    """A call without new tokens that only hands blocks on."""
    pool = phs.PagedPool(*(synth.normal_bf16((5, 2, 16, 64), s, device="cuda") for s in (1, 2)))
    a, b = phs.Int8Pool.empty(2, 2, 64), phs.Int8Pool.empty(2, 2, 64)
    none = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    table, qtable = dev([[4, 0, 2, 1, 3]]), dev([[1, 0]])
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    phs.kv_write_paged(pool, none, none, table, dev([70]), cu_seqlens=dev([0, 0]), int8=a,
                       qtable=qtable, qlens_before=dev([0]), qlens=dev([64]), max_qblocks=2,
                       status=st)
    phs.kv_quant_int8_block32(pool, table, b, qtable, dev([0]), dev([2]), 2, status=st)
    assert int(st.item()) == 0
    for x, y in ((a.k, b.k), (a.v, b.v), (a.k_scale, b.k_scale), (a.v_scale, b.v_scale)):
        assert torch.equal(x, y)
