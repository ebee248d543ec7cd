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
