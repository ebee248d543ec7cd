"""The selective scan against the token-by-token recurrence in 64 bits."""
import math

import numpy as np
import pytest
import torch

import layers_ref as ref
import paged_hybrid_sliding_gb300 as phs
import synth
from gpu_util import dev

pytestmark = pytest.mark.gpu


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


class Layer:
    def __init__(self, H, G, P, N, states, seed, plain=False):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.H, self.G, self.P, self.N = H, G, P, N
        step = torch.exp(torch.rand(H, generator=g, device="cuda") * math.log(100) + math.log(1e-3))
        self.w = phs.ScanWeights(
            -1 - 15 * torch.rand(H, generator=g, device="cuda"),
            None if plain else torch.randn(H, generator=g, device="cuda"),
            None if plain else step + torch.log(-torch.expm1(-step)))
        self.pool = phs.ScanPool(torch.randn((states, H, P, N), generator=g, device="cuda"))
        self.start = self.pool.s.clone()

    def inputs(self, T, seed, dt=torch.bfloat16, pad=8):
        H, G, P, N = self.H, self.G, self.P, self.N
        r = synth.normal_bf16((T, H * P + 2 * G * N + pad), seed, device="cuda")
        x, b, c = r[:, pad:].split([H * P, G * N, G * N], 1)
        d = synth.normal_bf16((T, H + 3), seed + 1, device="cuda")[:, 3:].to(dt)
        return (x.unflatten(1, (H, P)), d if dt == torch.bfloat16 else d * 0.7,
                b.unflatten(1, (G, N)), c.unflatten(1, (G, N)))

    def check(self, ins, out, spans, ids, resume, chunked):
        left = set(range(self.start.shape[0]))
        for i, (lo, hi) in enumerate(spans):
            if ids[i] < 0:
                assert not out[lo:hi].any()
                continue
            left.discard(int(ids[i]))
            s = self.start[ids[i]]
            if resume is not None and not resume[i]:
                s = torch.zeros_like(s)
            y, S, m, A, log = ref.scan(*(t[lo:hi] for t in ins), s, self.w.rate, self.w.skip,
                                       self.w.dt_bias)
            bo, bs = ref.scan_bounds(y, m, A, log, out.dtype, self.N, chunked)
            ref.close(out[lo:hi], y, bo, f"out {i}")
            ref.close(self.pool.s[ids[i]], S, bs, f"state {i}")
        left = sorted(left)
        assert torch.equal(self.pool.s[left], self.start[left])


SHAPES = [(1, 1, 64, 64), (3, 1, 64, 128), (4, 2, 64, 64), (6, 2, 64, 128), (2, 2, 128, 128),
          (4, 1, 128, 64), (8, 8, 64, 128)]


@pytest.mark.parametrize("H,G,P,N", SHAPES)
@pytest.mark.parametrize("dtype,dt", [(torch.float32, torch.bfloat16),
                                      (torch.bfloat16, torch.float32)])
def test_decode(H, G, P, N, dtype, dt):
    L = Layer(H, G, P, N, 9, H, plain=H == 4)
    ids = np.array([7, 0, -1, 3, 8])
    ins = L.inputs(5, 1, dt)
    st = status()
    out = phs.selective_scan_decode(*ins, L.pool, L.w, state_ids=dev(ids), out_dtype=dtype,
                                    status=st)
    assert int(st.item()) == 0 and out.dtype == dtype
    L.check(ins, out, [(b, b + 1) for b in range(5)], ids, None, False)


def test_decode_of_extreme_steps():
    """Steps of zero, of a strong decay, and far above softplus's bend."""
    L = Layer(4, 1, 64, 64, 3, 1)
    L.w.dt_bias[:] = torch.tensor([-200.0, 30.0, 0.0, 1e4])
    L.w.rate[:] = torch.tensor([-1.0, -4.0, 0.0, -1e30])
    ins = L.inputs(3, 5)
    out = phs.selective_scan_decode(*ins, L.pool, L.w, out_dtype=torch.float32)
    L.check(ins, out, [(0, 1), (1, 2), (2, 3)], np.arange(3), None, False)
    assert torch.equal(L.pool.s[:, 0], L.start[:, 0])   # exp(-200) x b is below every state's step


LENS = [[1], [0, 5, 0], [127, 128, 129], [64, 3, 63, 65, 1, 300], [1000], [17, 2, 256, 0, 640]]


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("H,G,P,N", SHAPES)
def test_prompt(lens, H, G, P, N):
    B = len(lens)
    L = Layer(H, G, P, N, B + 2, B, plain=H == 4)
    rng = np.random.default_rng(B)
    ids, resume = rng.permutation(B + 2)[:B], rng.integers(0, 2, B)
    if B > 3:
        ids[1] = -5
    cu = np.concatenate([[3], 3 + np.cumsum(lens)])   # rows of no request before and behind
    T = int(cu[-1]) + 2
    ins = L.inputs(T, 11, torch.float32 if H == 6 else torch.bfloat16)
    out = torch.full((T, H, P), 2.0, dtype=torch.bfloat16, device="cuda")
    st = status()
    assert phs.selective_scan_prompt(*ins, dev(cu), max(lens), L.pool, L.w, state_ids=dev(ids),
                                     resume=dev(resume), out=out, status=st) is out
    assert int(st.item()) == 0
    L.check(ins, out, list(zip(cu[:-1], cu[1:])), ids, resume, True)
    assert bool((out[:3] == 2).all()) and bool((out[cu[-1]:] == 2).all())


@pytest.mark.parametrize("H,G,P,N,n", [(2, 1, 64, 128, 5000), (24, 8, 64, 64, 1500),
                                       (40, 1, 64, 128, 700), (3, 3, 128, 128, 2500)])
def test_long_prompts(H, G, P, N, n):
    """Prompts that are cut into segments, and more heads than SMs can hold at once."""
    L = Layer(H, G, P, N, 3, H)
    ins = L.inputs(n + 300, 3)
    out = phs.selective_scan_prompt(*ins, dev([0, n, n + 300]), n, L.pool, L.w,
                                    state_ids=dev([2, 0]), resume=dev([1, 0]))
    L.check(ins, out, [(0, n), (n, n + 300)], [2, 0], [1, 0], True)


@pytest.mark.parametrize("rate,bias", [(-1e-4, 0.0), (0.0, 1.0), (-1e3, 3.0), (-0.01, -8.0),
                                       (-1e30, 5.0)])
def test_decay_extremes(rate, bias):
    """Memories of thousands of tokens, of none, and no decay at all."""
    L = Layer(2, 1, 64, 64, 2, 3)
    L.w.rate[:], L.w.dt_bias[:] = rate, bias
    ins = L.inputs(700, 5)
    out = phs.selective_scan_prompt(*ins, dev([0, 400, 700]), 400, L.pool, L.w, resume=dev([1, 1]))
    L.check(ins, out, [(0, 400), (400, 700)], [0, 1], [1, 1], True)


def test_steps_of_very_different_size():
    """A chunk whose tokens decay by next to nothing and by everything in turn."""
    L = Layer(2, 2, 64, 128, 1, 3)
    ins = list(L.inputs(300, 5, torch.float32))
    ins[1] = ins[1] * 6
    ins[1][::37] = 40.0
    ins[1][5::41] = -60.0
    out = phs.selective_scan_prompt(*ins, dev([0, 300]), 300, L.pool, L.w, resume=dev([1]))
    L.check(ins, out, [(0, 300)], [0], [1], True)


def test_prompt_in_parts_then_tokens():
    H, G, P, N = 4, 1, 64, 128
    L = Layer(H, G, P, N, 1, 9)
    ins = L.inputs(400, 7)
    got, at = [], 0
    for n in (1, 130, 257, 6):
        got.append(phs.selective_scan_prompt(*(t[at:at + n] for t in ins), dev([0, n]), n, L.pool,
                                             L.w, resume=dev([1])))
        at += n
    for t in range(at, 400):
        got.append(phs.selective_scan_decode(*(x[t:t + 1] for x in ins), L.pool, L.w))
    L.check(ins, torch.cat(got), [(0, 400)], [0], [1], True)


@pytest.mark.parametrize("H,G,P,N", SHAPES)
@pytest.mark.parametrize("lens", [[16], [1, 2, 15, 16, 0, 7], [17, 16, 1, 0, 200, 8, 5],
                                  [16, 16, 300, 16]])
def test_short_requests_are_their_tokens(lens, H, G, P, N):
    """Requests of up to 16 tokens give bit for bit what their tokens give one
    by one, beside longer ones too."""
    B = len(lens)
    L, M = (Layer(H, G, P, N, B + 2, B, plain=H == 4) for _ in range(2))
    rng = np.random.default_rng(H + B)
    ids, resume = rng.permutation(B + 2)[:B], rng.integers(0, 2, B)
    ids[B - 1] = -1 if B > 4 else ids[B - 1]
    cu = np.concatenate([[2], 2 + np.cumsum(lens)])
    T = int(cu[-1]) + 1
    ins = L.inputs(T, 11, torch.float32 if H == 6 else torch.bfloat16)
    out, st = torch.full((T, H, P), 2.0, dtype=torch.bfloat16, device="cuda"), status()
    phs.selective_scan_prompt(*ins, dev(cu), max(lens), L.pool, L.w, state_ids=dev(ids),
                              resume=dev(resume), out=out, status=st)
    assert int(st.item()) == 0
    L.check(ins, out, list(zip(cu[:-1], cu[1:])), ids, resume, True)
    assert bool((out[:2] == 2).all()) and bool((out[-1:] == 2).all())
    for b, n in enumerate(lens):
        if n > 16 or ids[b] < 0:
            continue
        if not resume[b]:
            M.pool.s[ids[b]] = 0
        for t in range(int(cu[b]), int(cu[b + 1])):
            one = phs.selective_scan_decode(*(x[t:t + 1] for x in ins), M.pool, M.w,
                                            state_ids=dev([ids[b]]))
            assert torch.equal(out[t], one[0]), (b, t)
        assert torch.equal(L.pool.s[ids[b]], M.pool.s[ids[b]]), b


@pytest.mark.parametrize("rate,bias", [(-1e-4, 0.0), (0.0, 1.0), (-1e3, 3.0), (-0.01, -8.0),
                                       (-1e30, 5.0)])
def test_decay_extremes_of_short_requests(rate, bias):
    L = Layer(2, 1, 64, 64, 3, 3)
    L.w.rate[:], L.w.dt_bias[:] = rate, bias
    ins = L.inputs(30, 5)
    out = phs.selective_scan_prompt(*ins, dev([0, 16, 25, 30]), 16, L.pool, L.w,
                                    resume=dev([1, 0, 1]))
    L.check(ins, out, [(0, 16), (16, 25), (25, 30)], [0, 1, 2], [1, 0, 1], True)


def test_bad_short_requests():
    """A bad range, a state that an earlier request has, one outside the pool:
    refused in the short requests' launch as in the others'."""
    H, G, P, N = 2, 1, 64, 64
    L = Layer(H, G, P, N, 4, 1)
    ins = L.inputs(40, 3)
    for extra, most in ((0, 16), (24, 300)):     # alone, and beside a longer request
        L.pool.s.copy_(L.start)
        out, st = torch.full((40, H, P), 2.0, dtype=torch.bfloat16, device="cuda"), status()
        phs.selective_scan_prompt(*ins, dev([0, 5, 9, 16, 16 + extra]), most, L.pool, L.w,
                                  state_ids=dev([1, 1, 7, 0]), out=out, status=st)
        assert int(st.item()) in (-1, -3) and not out[5:16].any()
        assert torch.equal(L.pool.s[[2, 3]], L.start[[2, 3]])
        assert bool((out[16 + extra:] == 2).all()) and bool((out[:5] != 2).any())
        L.pool.s.copy_(L.start)
        out.fill_(2)
        phs.selective_scan_prompt(*ins, dev([0, 12, 6, 16, 16 + extra]), most, L.pool, L.w,
                                  state_ids=dev([1, 2, 3, 0]), out=out, status=st)
        assert torch.equal(L.pool.s[[2, 3]], L.start[[2, 3]])
        assert bool((out[12:16] == 2).all())


def test_values_that_are_not_finite_stay_in_their_request():
    H, G, P, N = 2, 1, 64, 64
    L, M = Layer(H, G, P, N, 3, 1), Layer(H, G, P, N, 3, 1)
    ins = L.inputs(600, 3)
    cu = dev([0, 200, 400, 600])
    want = phs.selective_scan_prompt(*ins, cu, 200, M.pool, M.w)
    bad = [t.clone() for t in ins]
    bad[0][210, 0, 3], bad[2][390, 0, 5], bad[3][260, 0, 1] = float("nan"), float("inf"), float("nan")
    out = phs.selective_scan_prompt(*bad, cu, 200, L.pool, L.w)
    for lo, hi in ((0, 200), (400, 600)):
        assert torch.equal(out[lo:hi], want[lo:hi])
    assert torch.equal(L.pool.s[[0, 2]], M.pool.s[[0, 2]])
    assert torch.isnan(out[399, 0, 3]) and torch.isnan(L.pool.s[1, 0, 3]).all()


def test_bad_ranges_and_lengths():
    H, G, P, N = 2, 1, 64, 64
    for cu, most, refused in (([0, 200, 100, 300], 300, [1, 2]), ([0, 100, 200, 300], 99, [0, 1, 2]),
                              ([-1, 100, 200, 300], 300, [0]), ([0, 100, 200, 301], 300, [2])):
        L = Layer(H, G, P, N, 3, 1)
        ins = L.inputs(300, 3)
        out = torch.full((300, H, P), 2.0, dtype=torch.bfloat16, device="cuda")
        st = status()
        phs.selective_scan_prompt(*ins, dev(cu), most, L.pool, L.w, out=out, status=st)
        assert int(st.item()) == -3
        for b in range(3):
            lo, hi = cu[b], cu[b + 1]
            if b in refused:
                assert torch.equal(L.pool.s[b], L.start[b])
            else:
                y, S, m, A, log = ref.scan(*(t[lo:hi] for t in ins), torch.zeros_like(L.start[b]),
                                           L.w.rate, L.w.skip, L.w.dt_bias)
                bo, bs = ref.scan_bounds(y, m, A, log, out.dtype, N, True)
                ref.close(out[lo:hi], y, bo, f"out {b}")
                ref.close(L.pool.s[b], S, bs, f"state {b}")


def test_bad_states():
    H, G, P, N = 2, 1, 64, 64
    for ids, code, refused in (([2, 9, 1], -3, [1]), ([2, 2, 2], -1, [1, 2]), ([0, -7, -7], 0, [1, 2])):
        own = np.array([-1 if b in refused else i for b, i in enumerate(ids)])
        L = Layer(H, G, P, N, 4, 1)
        ins = L.inputs(270, 3)
        st = status()
        out = phs.selective_scan_prompt(*ins, dev([0, 130, 135, 270]), 135, L.pool, L.w,
                                        state_ids=dev(ids), status=st)
        assert int(st.item()) == code
        L.check(ins, out, [(0, 130), (130, 135), (135, 270)], own, [0, 0, 0], True)
        L = Layer(H, G, P, N, 4, 1)
        ins = L.inputs(3, 3)
        st = status()
        out = phs.selective_scan_decode(*ins, L.pool, L.w, state_ids=dev(ids), status=st)
        assert int(st.item()) == code
        L.check(ins, out, [(0, 1), (1, 2), (2, 3)], own, None, False)


def test_refusals_of_the_binding():
    L = Layer(4, 2, 64, 64, 3, 1)
    x, dt, b, c = L.inputs(3, 1)
    w = L.w
    for bad in (dict(x=x.float()), dict(x=x[:, :2]), dict(x=x.transpose(0, 1)), dict(dt=dt[:, :3]),
                dict(dt=dt.half()), dict(b=b[:2]), dict(b=b[..., :32], c=c[..., :32]), dict(c=c[:, :1]),
                dict(ids=dev([0])), dict(out=x[:2]), dict(w=phs.ScanWeights(w.rate[:2])),
                dict(w=phs.ScanWeights(w.rate, w.skip[:2])),
                dict(w=phs.ScanWeights(w.rate, None, w.rate.double())), dict(x=x.cpu())):
        a = dict(x=x, dt=dt, b=b, c=c, w=w, ids=None, out=None) | bad
        with pytest.raises((ValueError, TypeError)):
            phs.selective_scan_decode(a["x"], a["dt"], a["b"], a["c"], L.pool, a["w"],
                                      state_ids=a["ids"], out=a["out"])
    with pytest.raises(phs.PhsError):      # three groups do not divide four heads
        y = torch.zeros((3, 3, 64), dtype=torch.bfloat16, device="cuda")
        phs.selective_scan_decode(x, dt, y, y, L.pool, w)
    ws = torch.empty(8, dtype=torch.uint8, device="cuda")
    with pytest.raises(phs.PhsError):
        phs.selective_scan_prompt(x, dt, b, c, dev([0, 3]), 3, L.pool, w, workspace=ws)
    assert torch.equal(L.pool.s, L.start)
