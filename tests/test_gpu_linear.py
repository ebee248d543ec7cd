"""Linear attention with a decay per head against the token-by-token
recurrence in 64 bits."""
import math

import numpy as np
import pytest
import torch

import ops_ref
import paged_hybrid_sliding_gb300 as phs
import synth
from gpu_util import dev

pytestmark = pytest.mark.gpu


def decays(heads, lo=2e-4, hi=0.7):
    return -torch.logspace(math.log10(hi), math.log10(lo), heads, device="cuda")


def state_pool(n, heads, D, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return phs.StatePool(torch.randn((n, heads, D, D), generator=g, device="cuda"))


def bounds(ref, mag, state, smag, out_dtype, tokens, D):
    """A product of fp32 values and its addition round by 2^-24 each: a token
    adds at most 3 roundings to each state element (decay, product, sum) and
    the decay factor itself is off by 2^-22 (expf), all of the absolute sums:
    (tokens + 8) 2^-22 of the state's.  An output adds D products and, where
    tiles of tokens go through 16-bit matrix instructions, their operands are
    held to 16 bits or more: 2^-13 of its absolute sum covers the three such
    operands, and half a step of its own type."""
    rel = (tokens + 8) * 2.0**-22
    step = torch.finfo(out_dtype).eps / 2
    chunked = 2.0**-13 if out_dtype == torch.bfloat16 else 0.0
    return (mag * (rel + D * 2.0**-23 + chunked) + ref.abs() * step, smag * rel)


def close(got, ref, bound, what):
    err = (got.double() - ref).abs()
    assert torch.isfinite(got).all(), what
    assert bool((err <= bound).all()), \
        f"{what}: err {float(err.max()):.3e}, worst excess {float((err - bound).max()):.3e}"


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (4, 2), (6, 2), (5, 1), (16, 1), (32, 8)])
def test_decode(D, dtype, Hq, Hkv):
    B = 5
    pool = state_pool(9, Hkv, D, Hq)
    start = pool.s.clone()
    ids = np.array([7, 0, -1, 3, 8], np.int32)
    q = synth.normal_bf16((B, Hq, D), 1, device="cuda")
    k = synth.normal_bf16((B, Hkv, D), 2, device="cuda")
    v = synth.normal_bf16((B, Hkv, D), 3, device="cuda")
    g = decays(Hkv)
    g[0] = -math.inf                      # a head without memory
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = phs.linear_attn_decode(q, k, v, pool, g, state_ids=dev(ids), out_dtype=dtype, status=st)
    assert int(st.item()) == 0
    for b in range(B):
        if ids[b] < 0:
            assert not out[b].any()
            continue
        r, S, m, A = ops_ref.linear(q[b:b + 1], k[b:b + 1], v[b:b + 1], start[ids[b]], g,
                                    1 / math.sqrt(D))
        bo, bs = bounds(r, m, S, A, dtype, 1, D)
        close(out[b], r[0], bo[0], f"out {b}")
        close(pool.s[ids[b]], S, bs, f"state {b}")
    untouched = [i for i in range(9) if i not in ids]
    assert torch.equal(pool.s[untouched], start[untouched])


LENS = [[1], [0, 5, 0], [127, 128, 129], [64, 3, 63, 65, 1, 300], [1000], [17, 2, 256, 0, 640]]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (8, 2), (3, 1)])
@pytest.mark.parametrize("lens", LENS)
def test_prompt(D, Hq, Hkv, lens):
    B = len(lens)
    cu = np.concatenate([[2], 2 + np.cumsum(lens)]).astype(np.int32)
    T = int(cu[-1]) + 3                   # rows of no request in front and behind
    pool = state_pool(B + 2, Hkv, D, 4)
    start = pool.s.clone()
    ids = np.random.RandomState(B).permutation(B + 2)[:B].astype(np.int32)
    resume = np.arange(B) % 2
    q = synth.normal_bf16((T, Hq, D), 5, device="cuda")
    k = synth.normal_bf16((T, Hkv, D), 6, device="cuda")
    v = synth.normal_bf16((T, Hkv, D), 7, device="cuda")
    # what lies outside the requests must not reach them
    for t in (q, k, v):
        t[:2] = float("nan")
        t[T - 3:] = float("inf")
    g = decays(Hkv)
    out = torch.full((T, Hq, D), 3.0, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    phs.linear_attn_prompt(q, k, v, dev(cu), max(lens), pool, g, state_ids=dev(ids),
                           resume=dev(resume), out=out, status=st)
    assert int(st.item()) == 0
    assert (out[:2] == 3).all() and (out[T - 3:] == 3).all()
    for b in range(B):
        a, e = int(cu[b]), int(cu[b + 1])
        s0 = start[ids[b]] if resume[b] else torch.zeros_like(start[0])
        r, S, m, A = ops_ref.linear(q[a:e], k[a:e], v[a:e], s0, g, 1 / math.sqrt(D))
        bo, bs = bounds(r, m, S, A, torch.bfloat16, e - a, D)
        close(out[a:e], r, bo, f"out of request {b}")
        close(pool.s[ids[b]], S, bs, f"state of request {b}")
    rest = [i for i in range(B + 2) if i not in ids]
    assert torch.equal(pool.s[rest], start[rest])


def test_long_prompt_few_heads():
    D, T = 128, 5003
    pool = state_pool(1, 2, D, 8)
    q = synth.normal_bf16((T, 2, D), 9, device="cuda")
    k = synth.normal_bf16((T, 2, D), 10, device="cuda")
    v = synth.normal_bf16((T, 2, D), 11, device="cuda")
    g = decays(2, lo=1e-5, hi=0.02)
    out = phs.linear_attn_prompt(q, k, v, dev([0, T]), T, pool, g)
    r, S, m, A = ops_ref.linear(q, k, v, torch.zeros((2, D, D), device="cuda"), g,
                                1 / math.sqrt(D))
    bo, bs = bounds(r, m, S, A, torch.bfloat16, T, D)
    close(out, r, bo, "out")
    close(pool.s[0], S, bs, "state")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,lens", [
    (16, 1, [1100]),                 # segments, and the heads of a group on several CTAs
    (6, 1, [700, 0, 1, 1300]),       # requests of one segment and of none beside longer ones
    (12, 4, [200, 129]),             # groups of heads, no segments
    (8, 8, [2100]), (5, 1, [515, 513])])
def test_segments_and_groups_of_heads(D, Hq, Hkv, lens):
    B = len(lens)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T = int(cu[-1])
    q = synth.normal_bf16((T, Hq, D), 31, device="cuda")
    k = synth.normal_bf16((T, Hkv, D), 32, device="cuda")
    v = synth.normal_bf16((T, Hkv, D), 33, device="cuda")
    g = decays(Hkv, lo=1e-3)
    for resume in ([1] * B, [0] * B, [r % 2 for r in range(B)], None):
        pool = state_pool(B, Hkv, D, 34)
        start = pool.s.clone()
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = phs.linear_attn_prompt(q, k, v, dev(cu), max(lens), pool, g,
                                     resume=None if resume is None else dev(resume), status=st)
        assert int(st.item()) == 0
        for b in range(B):
            a, e = int(cu[b]), int(cu[b + 1])
            s0 = start[b] if resume and resume[b] else torch.zeros_like(start[b])
            r, S, m, A = ops_ref.linear(q[a:e], k[a:e], v[a:e], s0, g, 1 / math.sqrt(D))
            bo, bs = bounds(r, m, S, A, torch.bfloat16, e - a, D)
            close(out[a:e], r, bo, f"out of request {b}")
            close(pool.s[b], S, bs, f"state of request {b}")


@pytest.mark.parametrize("value", [0.0, -1e-7, -3.0, -80.0, -1e6, -math.inf])
def test_prompt_decay_extremes(value):
    D, T = 64, 200
    pool = state_pool(1, 1, D, 12)
    s0 = pool.s[0].clone()
    q = synth.normal_bf16((T, 1, D), 13, device="cuda")
    k = synth.normal_bf16((T, 1, D), 14, device="cuda")
    v = synth.normal_bf16((T, 1, D), 15, device="cuda")
    g = torch.full((1,), value, device="cuda")
    out = phs.linear_attn_prompt(q, k, v, dev([0, T]), T, pool, g, resume=dev([1]))
    r, S, m, A = ops_ref.linear(q, k, v, s0, g, 1 / math.sqrt(D))
    bo, bs = bounds(r, m, S, A, torch.bfloat16, T, D)
    close(out, r, bo, "out")
    close(pool.s[0], S, bs, "state")


@pytest.mark.parametrize("B", [40, 256, 257])
def test_many_short_prompts(B):
    """More CTAs than SMs, with and without an order by length."""
    D, Hq, Hkv = 64, 8, 4
    lens = np.random.RandomState(B).randint(0, 180, B)
    lens[B // 2], lens[B // 3] = 700, 0
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T = int(cu[-1])
    q = synth.normal_bf16((T, Hq, D), 35, device="cuda")
    k = synth.normal_bf16((T, Hkv, D), 36, device="cuda")
    v = synth.normal_bf16((T, Hkv, D), 37, device="cuda")
    g = decays(Hkv, lo=1e-3)
    pool = state_pool(B, Hkv, D, 38)
    start = pool.s.clone()
    ids = np.random.RandomState(1).permutation(B).astype(np.int32)
    ids[5] = -1
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = phs.linear_attn_prompt(q, k, v, dev(cu), 700, pool, g, state_ids=dev(ids),
                                 resume=dev(np.arange(B) % 2), status=st)
    assert int(st.item()) == 0
    assert not out[cu[5]:cu[6]].any()
    for b in [b for b in range(B) if b != 5 and (b < 12 or b > B - 6 or lens[b] in (0, 700))]:
        a, e = int(cu[b]), int(cu[b + 1])
        s0 = start[ids[b]] if b % 2 else torch.zeros_like(start[0])
        r, S, m, A = ops_ref.linear(q[a:e], k[a:e], v[a:e], s0, g, 1 / math.sqrt(D))
        bo, bs = bounds(r, m, S, A, torch.bfloat16, e - a, D)
        close(out[a:e], r, bo, f"out of request {b}")
        close(pool.s[ids[b]], S, bs, f"state of request {b}")
    # the others against calls of their own
    for b in range(12, B - 6, 7):
        a, e = int(cu[b]), int(cu[b + 1])
        one = phs.StatePool(start[ids[b]][None].clone())
        ref = phs.linear_attn_prompt(q[a:e], k[a:e], v[a:e], dev([0, e - a]), max(e - a, 1), one,
                                     g, resume=dev([b % 2]))
        assert torch.allclose(out[a:e].float(), ref.float(), rtol=2**-7, atol=1e-3)


def test_prompt_in_parts_then_decode_is_one_prompt():
    """A prompt in two calls, then single tokens, against one recurrence."""
    D, Hq, Hkv, T = 128, 4, 2, 391
    q = synth.normal_bf16((T, Hq, D), 16, device="cuda")
    k = synth.normal_bf16((T, Hkv, D), 17, device="cuda")
    v = synth.normal_bf16((T, Hkv, D), 18, device="cuda")
    g = decays(Hkv)
    pool = state_pool(3, Hkv, D, 19)      # stale states: the first part starts from zero
    ids = dev([1])
    outs = []
    for a, e, go in ((0, 200, 0), (200, 385, 1)):
        outs.append(phs.linear_attn_prompt(q[a:e], k[a:e], v[a:e], dev([0, e - a]), e - a, pool, g,
                                           state_ids=ids, resume=dev([go])))
    for t in range(385, T):
        outs.append(phs.linear_attn_decode(q[t:t + 1], k[t:t + 1], v[t:t + 1], pool, g,
                                           state_ids=ids))
    r, S, m, A = ops_ref.linear(q, k, v, torch.zeros((Hkv, D, D), device="cuda"), g,
                                1 / math.sqrt(D))
    bo, bs = bounds(r, m, S, A, torch.bfloat16, T, D)
    close(torch.cat(outs), r, bo, "out")
    close(pool.s[1], S, bs, "state")


def test_bad_ids_and_ranges():
    D, H = 64, 2
    q = synth.normal_bf16((4, H, D), 20, device="cuda")
    g = decays(H)
    for bad, code in (([0, 9, 1, 2], -3), ([2, 0, 2, 1], -1)):
        pool = state_pool(3, H, D, 21)
        ref = phs.StatePool(pool.s.clone())
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = phs.linear_attn_decode(q, q, q, pool, g, state_ids=dev(bad), status=st)
        assert int(st.item()) == code
        skip = 1 if code == -3 else 2
        assert not out[skip].any()
        keep = [b for b in range(4) if b != skip]
        good = phs.linear_attn_decode(q[keep], q[keep], q[keep], ref, g,
                                      state_ids=dev([bad[b] for b in keep]))
        assert torch.equal(out[keep], good) and torch.equal(pool.s, ref.s)
    # prompts: a bad range, one longer than stated, a repeated and an inactive state
    q = synth.normal_bf16((100, H, D), 22, device="cuda")
    for cu, ids, most, code, zero, kept in (
            ([0, 40, 30, 100], [0, 1, 2], 70, -3, [], [(0, 40)]),
            ([0, 40, 100, 200], [0, 1, 2], 60, -3, [], [(0, 40), (40, 100)]),
            ([0, 10, 90, 100], [0, 1, 2], 50, -3, [], [(0, 10), (90, 100)]),
            ([0, 10, 90, 100], [0, 0, 2], 80, -1, [(10, 90)], [(0, 10), (90, 100)]),
            ([0, 10, 90, 100], [0, -1, 2], 80, 0, [(10, 90)], [(0, 10), (90, 100)])):
        pool = state_pool(3, H, D, 23)
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full((100, H, D), 5.0, dtype=torch.bfloat16, device="cuda")
        phs.linear_attn_prompt(q, q, q, dev(cu), most, pool, g, state_ids=dev(ids), out=out,
                               status=st)
        assert int(st.item()) == code, cu
        for a, e in zero:
            assert not out[a:e].any()
        done = torch.zeros(100, dtype=torch.bool)
        for a, e in zero + kept:
            done[a:e] = True
        assert (out[~done] == 5).all()
        for a, e in kept:
            one = state_pool(1, H, D, 24)
            ref = phs.linear_attn_prompt(q[a:e], q[a:e], q[a:e], dev([0, e - a]), e - a, one, g)
            assert torch.allclose(out[a:e].float(), ref.float(), rtol=2**-7, atol=1e-3)


def test_graph_and_side_stream():
    D, H, T = 128, 4, 300
    q = synth.normal_bf16((T, H, D), 25, device="cuda")
    k = synth.normal_bf16((T, H, D), 26, device="cuda")
    v = synth.normal_bf16((T, H, D), 27, device="cuda")
    g = decays(H)
    pool = state_pool(2, H, D, 28)
    s0 = pool.s.clone()
    cu = dev([0, 170, T])
    need = phs.linear_prompt_workspace_bytes(2, H, H, D, T, 170)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    d_out = torch.empty((2, H, D), dtype=torch.bfloat16, device="cuda")
    resume = dev([1, 1])

    def step(stream=None):
        phs.linear_attn_prompt(q, k, v, cu, 170, pool, g, resume=resume, out=out, workspace=ws,
                               stream=stream)
        phs.linear_attn_decode(q[:2], k[:2], v[:2], pool, g, out=d_out, stream=stream)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    step(s)
    s.synchronize()
    want = [out.clone(), d_out.clone(), pool.s.clone()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    pool.s.copy_(s0)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(want, (out, d_out, pool.s)):
        assert torch.equal(x, y)


def test_refusals():
    D, H = 64, 2
    pool = state_pool(2, H, D, 29)
    g = decays(H)
    q = synth.normal_bf16((2, H, D), 30, device="cuda")
    with pytest.raises(phs.PhsError) as e:      # more requests than states
        phs.linear_attn_decode(q.repeat(2, 1, 1), q.repeat(2, 1, 1), q.repeat(2, 1, 1), pool, g)
    assert e.value.code == -2
    with pytest.raises(phs.PhsError) as e:
        phs.linear_attn_decode(q, q, q, pool, g, scale=float("inf"))
    assert e.value.code == -1
    with pytest.raises(phs.PhsError) as e:      # three query heads on two states
        phs.linear_attn_decode(synth.normal_bf16((2, 3, D), 1, device="cuda"), q, q, pool, g)
    assert e.value.code == -2
    wide = phs.StatePool(torch.zeros((2, H, 96, 96), device="cuda"))
    x = synth.normal_bf16((2, H, 96), 1, device="cuda")
    with pytest.raises(phs.PhsError) as e:
        phs.linear_attn_decode(x, x, x, wide, g)
    assert e.value.code == -7
    with pytest.raises(phs.PhsError) as e:
        phs.linear_attn_prompt(q, q, q, dev([0, 2]), 2, pool, g,
                               workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    assert e.value.code == -5
    for bad in (lambda: phs.linear_attn_decode(q, q[:1], q, pool, g),
                lambda: phs.linear_attn_decode(q, q, q, pool, g.double()),
                lambda: phs.linear_attn_decode(q, q, q, pool, g[:1]),
                lambda: phs.linear_attn_decode(q, q, q, pool, g, state_ids=dev([0])),
                lambda: phs.linear_attn_decode(q[:, :, ::2], q, q, pool, g),
                lambda: phs.linear_attn_prompt(q, q, q, dev([0, 2]), 2, pool, g,
                                               resume=dev([1, 1])),
                lambda: phs.linear_attn_prompt(q, q, q, dev([0, 2]), 2, pool, g,
                                               out=torch.empty_like(q, dtype=torch.float32))):
        with pytest.raises(ValueError):
            bad()
    # nothing to do
    e = q[:0]
    assert phs.linear_attn_decode(e, e, e, pool, g, state_ids=dev([])).shape[0] == 0
    phs.linear_attn_prompt(e, e, e, dev([0, 0]), 0, pool, g)
    phs.linear_attn_prompt(e, e, e, dev([0]), 0, pool, g, state_ids=dev([]))
