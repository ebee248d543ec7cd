"""Linear attention where it can go wrong: what lies behind a request's last
token, and decays that leave next to nothing of a state."""
import math

import numpy as np
import pytest
import torch

import ops_ref
import paged_hybrid_sliding_gb300 as phs
import synth
from gpu_util import dev
from test_gpu_linear import bounds, close, decays, state_pool

pytestmark = pytest.mark.gpu


def reference(q, k, v, start, g):
    D = q.shape[2]
    r, S, m, A = ops_ref.linear(q, k, v, start, g, 1 / math.sqrt(D))
    return (r, S) + bounds(r, m, S, A, torch.bfloat16, q.shape[0], D)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("value", ["nan", "inf"])
@pytest.mark.parametrize("Hq,Hkv,chunks", [(2, 2, 0), (2, 2, 2), (4, 1, 1), (16, 8, 0)])
def test_a_bad_neighbour_does_not_reach_a_request(D, value, Hq, Hkv, chunks):
    """Requests that end at any place of a chunk, each followed by one that is
    infinite or NaN throughout, in q, k and v: outputs and states of the good ones
    are those of the recurrence, and the same every time."""
    last = [1, 17, 33, 44, 65, 70, 81, 104, 128]
    lens = [n for r in last for n in (chunks * 128 + r, 130)]
    B = len(lens)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T = int(cu[-1])
    q = synth.normal_bf16((T, Hq, D), 41, device="cuda")
    k = synth.normal_bf16((T, Hkv, D), 42, device="cuda")
    v = synth.normal_bf16((T, Hkv, D), 43, device="cuda")
    for b in range(1, B, 2):
        for t in (q, k, v):
            t[int(cu[b]):int(cu[b + 1])] = float(value)
    g = decays(Hkv)
    resume = np.arange(B) // 2 % 2
    pool = state_pool(B, Hkv, D, 44)
    start = pool.s.clone()
    first = None
    for _ in range(6):
        pool.s.copy_(start)
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = phs.linear_attn_prompt(q, k, v, dev(cu), max(lens), pool, g, resume=dev(resume),
                                     status=st)
        assert int(st.item()) == 0
        good = [out[int(cu[b]):int(cu[b + 1])].clone() for b in range(0, B, 2)]
        states = pool.s[::2].clone()
        if first is None:
            first = good, states
            for i, b in enumerate(range(0, B, 2)):
                a, e = int(cu[b]), int(cu[b + 1])
                s0 = start[b] if resume[b] else torch.zeros_like(start[b])
                r, S, bo, bs = reference(q[a:e], k[a:e], v[a:e], s0, g)
                close(good[i], r, bo, f"out of a request of {lens[b]} tokens")
                close(states[i], S, bs, f"state of a request of {lens[b]} tokens")
        else:
            assert all(torch.equal(x, y) for x, y in zip(good, first[0]))
            assert torch.equal(states, first[1])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [641, 705, 1000])
def test_a_chunk_of_bad_rows_behind_a_prompt_in_segments(D, n):
    """A prompt that is cut into segments, and a whole chunk of rows of no
    request behind it."""
    T, H = n + 130, 2
    q, k, v = (synth.normal_bf16((T, H, D), s, device="cuda") for s in (45, 46, 47))
    for t in (q, k, v):
        t[n:] = float("nan")
    g = decays(H, lo=1e-3)
    pool = state_pool(1, H, D, 48)
    start = pool.s[0].clone()
    out = torch.full((T, H, D), 3.0, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    phs.linear_attn_prompt(q, k, v, dev([0, n]), n, pool, g, resume=dev([1]), out=out, status=st)
    assert int(st.item()) == 0 and (out[n:] == 3).all()
    r, S, bo, bs = reference(q[:n], k[:n], v[:n], start, g)
    close(out[:n], r, bo, "out")
    close(pool.s[0], S, bs, "state")


# A state that strongly decays is exp(g n) of itself, not what is left of it after
# 1 - (1 - exp(g n)) has been rounded: at g n = -12 half a step of fp32 below 1 is
# 0.5 % of exp(g n).  The bounds are those of the other tests: some 2^-22 a token of
# the decayed absolute sums.  exp(g n) stays far above the smallest fp32 numbers.
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(8, 8), (24, 8)])
def test_decode_keeps_what_a_strong_decay_leaves(D, Hq, Hkv):
    pool = state_pool(3, Hkv, D, 51)
    start = pool.s.clone()
    q, k, v = (synth.normal_bf16((3, h, D), s, device="cuda")
               for h, s in ((Hq, 52), (Hkv, 53), (Hkv, 54)))
    k[:2] = 0                                # nothing comes in
    k[2] *= 2.0**-40                         # next to nothing
    g = -torch.tensor([0.3, 0.6, 1.0, 3.0, 8.0, 12.0, 20.0, 50.0], device="cuda")
    out = phs.linear_attn_decode(q, k, v, pool, g, out_dtype=torch.float32)
    for b in range(3):
        r, S, m, A = ops_ref.linear(q[b:b + 1], k[b:b + 1], v[b:b + 1], start[b], g,
                                    1 / math.sqrt(D))
        bo, bs = bounds(r, m, S, A, torch.float32, 1, D)
        close(out[b], r[0], bo[0], f"out {b}")
        close(pool.s[b], S, bs, f"state {b}")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [1, 100, 128, 200, 300])
def test_prompt_keeps_what_a_strong_decay_leaves(D, T):
    """A padded prompt: keys of zero behind its first tokens, or from the start."""
    H = 6
    q, k, v = (synth.normal_bf16((2 * T, H, D), s, device="cuda") for s in (55, 56, 57))
    k[:T] = 0
    k[T + 2:] = 0
    g = -torch.tensor([1e-3, 6e-3, 0.03, 0.08, 0.15, 0.2], device="cuda")
    pool = state_pool(2, H, D, 58)
    start = pool.s.clone()
    out = phs.linear_attn_prompt(q, k, v, dev([0, T, 2 * T]), T, pool, g, resume=dev([1, 0]))
    for b in range(2):
        a, e = b * T, (b + 1) * T
        s0 = torch.zeros_like(start[0]) if b else start[0]
        r, S, bo, bs = reference(q[a:e], k[a:e], v[a:e], s0, g)
        close(out[a:e], r, bo, f"out {b}")
        close(pool.s[b], S, bs, f"state {b}")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [640, 1800])
def test_segments_keep_what_a_strong_decay_leaves(D, T):
    H = 2
    q, k, v = (synth.normal_bf16((T, H, D), s, device="cuda") for s in (59, 60, 61))
    k[:] = 0
    g = -torch.tensor([20 / T, 58 / T], device="cuda")
    pool = state_pool(1, H, D, 62)
    start = pool.s[0].clone()
    out = phs.linear_attn_prompt(q, k, v, dev([0, T]), T, pool, g, resume=dev([1]))
    r, S, bo, bs = reference(q, k, v, start, g)
    close(out, r, bo, "out")
    close(pool.s[0], S, bs, "state")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("value", ["nan", "inf"])
def test_how_far_a_bad_value_reaches(D, value):
    """An infinite or NaN row of v at token 300: the outputs of the chunks of 128
    tokens before its own, and of the other requests, are as without it; from its
    own on they are not finite."""
    H, T = 2, 500
    q, k, v = (synth.normal_bf16((2 * T, H, D), s, device="cuda") for s in (63, 64, 65))
    g = decays(H, lo=1e-3, hi=0.02)

    def run():
        pool = state_pool(2, H, D, 66)
        return phs.linear_attn_prompt(q, k, v, dev([0, T, 2 * T]), T, pool, g), pool.s

    out, s = run()
    v[300] = float(value)
    bad, bad_s = run()
    assert torch.equal(bad[:256], out[:256]) and torch.equal(bad[T:], out[T:])
    assert torch.equal(bad_s[1], s[1])
    assert not torch.isfinite(bad[300:T].float()).any() and not torch.isfinite(bad_s[0]).any()


@pytest.mark.parametrize("D", [64, 128])
def test_segments_beside_inactive_and_refused_requests(D):
    """Long prompts in segments, with a request without a state, one of a state
    that another has, one of a range beginning before the last one's end."""
    H, n = 1, 1400
    cu = [0, n, 2 * n, 3 * n, 4 * n, 4 * n - 300]
    ids = [2, -1, 2, 0, 1]
    T = 4 * n
    q, k, v = (synth.normal_bf16((T, H, D), s, device="cuda") for s in (67, 68, 69))
    g = decays(H, lo=1e-3, hi=1e-3)
    pool = state_pool(4, H, D, 70)
    start = pool.s.clone()
    out = torch.full((T, H, D), 3.0, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    phs.linear_attn_prompt(q, k, v, dev(cu), n, pool, g, state_ids=dev(ids),
                           resume=dev([1] * 5), out=out, status=st)
    assert int(st.item()) in (-1, -3)
    assert not out[n:3 * n].any()          # without a state, and of one that is taken
    for b, i in ((0, 2), (3, 0)):
        a, e = cu[b], cu[b + 1]
        r, S, bo, bs = reference(q[a:e], k[a:e], v[a:e], start[i], g)
        close(out[a:e], r, bo, f"out of request {b}")
        close(pool.s[i], S, bs, f"state {i}")
    assert torch.equal(pool.s[[1, 3]], start[[1, 3]])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(3, 3), (12, 2), (16, 1)])
def test_a_single_token_is_rounded_once(D, Hq, Hkv):
    """Its products are fp32 ones: a bf16 output is off by half a step of its own
    beside what the fp32 output is off by."""
    B = 4
    q, k, v = (synth.normal_bf16((B, h, D), s, device="cuda")
               for h, s in ((Hq, 71), (Hkv, 72), (Hkv, 73)))
    g = decays(Hkv)
    pool = state_pool(B, Hkv, D, 74)
    start = pool.s.clone()
    out = phs.linear_attn_decode(q, k, v, pool, g)
    for b in range(B):
        r, S, m, A = ops_ref.linear(q[b:b + 1], k[b:b + 1], v[b:b + 1], start[b], g,
                                    1 / math.sqrt(D))
        bo, _ = bounds(r, m, S, A, torch.float32, 1, D)
        close(out[b], r[0], (bo + (r.abs() + bo) * 2.0**-8)[0], f"out {b}")
