"""The causal convolution of a selective layer against its definition in 64
bits."""
import numpy as np
import pytest
import torch

import layers_ref as ref
import paged_hybrid_sliding_gb300 as phs
import synth
from gpu_util import dev

pytestmark = pytest.mark.gpu


def setup(C, W, states, seed, bias=True, silu=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = phs.ConvWeights(torch.randn((C, W), generator=g, device="cuda"),
                        torch.randn(C, generator=g, device="cuda") if bias else None, silu)
    pool = phs.ConvPool(synth.normal_bf16((states, W - 1, C), seed + 1, device="cuda"))
    return w, pool, pool.c.clone()


def rows(T, C, pad, seed):
    w = synth.normal_bf16((T, C + pad), seed, device="cuda")
    return w[:, pad:]


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def check(x, w, out, pool, start, spans, ids, resume):
    """spans: (first row, end) of each request."""
    left = set(range(pool.c.shape[0]))
    for b, (lo, hi) in enumerate(spans):
        if ids[b] < 0:
            assert not out[lo:hi].any()
            continue
        left.discard(int(ids[b]))
        old = start[ids[b]] if resume is None or resume[b] else torch.zeros_like(start[0])
        y, e, last = ref.conv(x[lo:hi], old, w.weight, w.bias, w.silu)
        ref.close(out[lo:hi], y, e, f"request {b}")
        assert torch.equal(pool.c[ids[b]], last), f"state {b}"
    left = sorted(left)
    assert torch.equal(pool.c[left], start[left])


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("C,pad,bias,silu", [(8, 0, True, True), (264, 8, False, True),
                                             (1280, 24, True, False), (4352, 4160, True, True)])
def test_decode(W, C, pad, bias, silu):
    B = 6
    w, pool, start = setup(C, W, B + 3, 3, bias, silu)
    ids = np.array([7, 0, -1, 3, 8, 5])
    x = rows(B, C, pad, 9)
    st = status()
    out = phs.causal_conv_decode(x, pool, w, state_ids=dev(ids), status=st)
    assert int(st.item()) == 0
    check(x, w, out, pool, start, [(b, b + 1) for b in range(B)], ids, None)
    # no ids: request b has state b
    w, pool, start = setup(C, W, B + 3, 3, bias, silu)
    phs.causal_conv_decode(x, pool, w, out=out)
    check(x, w, out, pool, start, [(b, b + 1) for b in range(B)], np.arange(B), None)


LENS = [[1], [0, 5, 0], [31, 1, 33], [1, 2, 3, 4, 1, 1, 0, 0, 2], [30, 3, 64, 2, 300],
        [32, 32, 0, 32], [1000]]


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("W,C,pad", [(4, 264, 8), (3, 64, 0), (2, 1280, 16), (4, 4352, 4160)])
def test_prompt(lens, W, C, pad):
    B = len(lens)
    w, pool, start = setup(C, W, B + 2, 5)
    rng = np.random.default_rng(B)
    ids, resume = rng.permutation(B + 2)[:B], rng.integers(0, 2, B)
    if B > 2:
        ids[1] = -5
    first = 3                                   # rows of no request before and behind
    cu = np.concatenate([[first], first + np.cumsum(lens)])
    T = int(cu[-1]) + 2
    x = rows(T, C, pad, 11)
    out = torch.full((T, C), 2.0, dtype=torch.bfloat16, device="cuda")
    st = status()
    assert phs.causal_conv_prompt(x, dev(cu), pool, w, state_ids=dev(ids), resume=dev(resume),
                                  out=out, status=st) is out
    assert int(st.item()) == 0
    check(x, w, out, pool, start, list(zip(cu[:-1], cu[1:])), ids, resume)
    assert bool((out[:first] == 2).all()) and bool((out[cu[-1]:] == 2).all())


def test_no_rows_at_all():
    """Requests without tokens: a state that is not continued becomes zero."""
    w, pool, start = setup(64, 4, 3, 1)
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    out = phs.causal_conv_prompt(x, dev([0, 0, 0]), pool, w, resume=dev([1, 0]))
    assert out.shape == (0, 64)
    assert torch.equal(pool.c[[0, 2]], start[[0, 2]]) and not pool.c[1].any()


@pytest.mark.parametrize("parts", [[100], [37, 63], [1, 1, 1, 97], [33, 1, 66], [2, 32, 66]])
def test_parts_give_what_the_whole_gives(parts):
    """A prompt in parts and then single tokens, bit for bit."""
    C = 264
    x = rows(104, C, 0, 13)
    w, pool, _ = setup(C, 4, 1, 7)
    pool.c.zero_()
    whole = phs.causal_conv_prompt(x, dev([0, 104]), phs.ConvPool(pool.c.clone()), w)
    got, at = [], 0
    for n in parts:
        got.append(phs.causal_conv_prompt(x[at:at + n], dev([0, n]), pool, w, resume=dev([1])))
        at += n
    for t in range(100, 104):
        got.append(phs.causal_conv_decode(x[t:t + 1], pool, w))
    assert torch.equal(torch.cat(got), whole)
    assert torch.equal(pool.c[0], x[101:])


def test_large_values():
    """Infinities and NaN stay where the filter puts them; silu of what
    overflows is 0 below and itself above."""
    C = 64
    w, pool, _ = setup(C, 2, 1, 1, bias=False)
    w.weight[:] = torch.tensor([0.0, 1.0])
    pool.c.zero_()
    x = torch.zeros((6, C), dtype=torch.bfloat16, device="cuda")
    x[0, 0], x[1, 0], x[2, 0] = 3e38, -3e38, -200.0
    x[3, 1], x[4, 2], x[5, 3] = float("inf"), float("-inf"), float("nan")
    w.weight[1:4, 0] = 1.0
    w.weight[4:, 0] = 0.0
    out = phs.causal_conv_prompt(x, dev([0, 6]), pool, w)
    assert float(out[0, 0]) == float(x[0, 0]) and float(out[1, 0]) == 0 and abs(float(out[2, 0])) < 1e-30
    assert float(out[3, 1]) == float("inf") and float(out[4, 1]) == float("inf")
    assert float(out[4, 2]) == 0 and float(out[5, 2]) == 0 and torch.isnan(out[5, 3])
    assert torch.isfinite(out[:, 4:]).all()


def test_bad_ranges_refuse_the_call():
    C = 64
    for cu in ([0, 20, 10, 40], [-1, 10, 20, 40], [0, 10, 20, 41]):
        w, pool, start = setup(C, 4, 3, 1)
        out = torch.full((40, C), 2.0, dtype=torch.bfloat16, device="cuda")
        st = status()
        phs.causal_conv_prompt(rows(40, C, 0, 1), dev(cu), pool, w, out=out, status=st)
        assert int(st.item()) == -3 and bool((out == 2).all()) and torch.equal(pool.c, start)


def test_bad_states():
    """An id outside the pool, one that an earlier request has."""
    C = 264
    for ids, code, refused in (([2, 9, 1], -3, [1]), ([2, 2, 2], -1, [1, 2]), ([0, -7, -7], 0, [1, 2])):
        w, pool, start = setup(C, 4, 4, 1)
        x = rows(70, C, 0, 1)
        st = status()
        out = phs.causal_conv_prompt(x, dev([0, 33, 35, 70]), pool, w, state_ids=dev(ids), status=st)
        assert int(st.item()) == code
        own = np.array([-1 if b in refused else i for b, i in enumerate(ids)])
        check(x, w, out, pool, start, [(0, 33), (33, 35), (35, 70)], own, [0, 0, 0])
        w, pool, start = setup(C, 4, 4, 1)
        st = status()
        out = phs.causal_conv_decode(x[:3], pool, w, state_ids=dev(ids), status=st)
        assert int(st.item()) == code
        check(x, w, out, pool, start, [(0, 1), (1, 2), (2, 3)], own, None)


def test_refusals_of_the_binding():
    w, pool, start = setup(64, 4, 3, 1)
    x = rows(5, 64, 0, 1)
    for bad in (dict(x=x.float()), dict(x=x[:, :56]), dict(x=x.t()), dict(x=x[:, ::2]),
                dict(ids=dev([0, 1])), dict(out=x[:3]), dict(x=x.cpu()),
                dict(w=phs.ConvWeights(w.weight[:, :3])), dict(w=phs.ConvWeights(w.weight.bfloat16())),
                dict(w=phs.ConvWeights(w.weight, w.bias[:8]))):
        a = dict(x=x, w=w, ids=None, out=None) | bad
        with pytest.raises((ValueError, TypeError)):
            phs.causal_conv_decode(a["x"], pool, a["w"], state_ids=a["ids"], out=a["out"])
    with pytest.raises(phs.PhsError):       # five requests, three states
        phs.causal_conv_decode(x, pool, w)
    with pytest.raises(phs.PhsError):       # rows that do not begin on 16 bytes
        phs.causal_conv_decode(rows(3, 64, 4, 1), pool, w)
    with pytest.raises(ValueError):
        phs.causal_conv_prompt(x, dev([]), pool, w)
    assert torch.equal(pool.c, start)


def test_a_token_over_its_own_input():
    C, W, B = 264, 4, 5
    w, pool, start = setup(C, W, B, 3, True, True)
    x = rows(B, C, 0, 9).contiguous()
    want = phs.causal_conv_decode(x, phs.ConvPool(start.clone()), w)
    phs.causal_conv_decode(x, pool, w, out=x)
    assert torch.equal(x, want)
