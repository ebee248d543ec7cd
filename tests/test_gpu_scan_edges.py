"""Prompts of the selective scan where they can go wrong unseen: workspaces past
32-bit counts, weights of single tokens, the order in which a call's requests
are taken, what a state keeps of its tokens."""
import math

import numpy as np
import pytest
import torch

import layers_ref as ref
import paged_hybrid_sliding_gb300 as phs
import synth
from gpu_util import dev
from test_gpu_scan import Layer

pytestmark = pytest.mark.gpu

CHUNK, TABLE = 128, 536


# ---------------------------------------------------------------- workspaces --
@pytest.mark.parametrize("B,H,P,N,total,most", [
    (65535, 128, 64, 64, 70_000, 100),          # 4.5e9 floats of tables
    (65535, 64, 64, 128, 65535 * 17, 17),       # 2.5e9: negative as a 32-bit number
    (2000, 4096, 64, 64, 34_000, 17),
    (16, 64, 64, 128, 32_000, 2000)])
def test_workspace_holds_a_table_for_each_chunk_and_head(B, H, P, N, total, most):
    """(The size alone: nothing is launched.)  Plans without segments hold the
    tables and nothing else, rounded up to 256 bytes."""
    want = (total // CHUNK + B + 1) * H * TABLE * 4
    got = phs.scan_prompt_workspace_bytes(B, H, 1, P, N, total, most)
    assert want <= got <= want + 256


# --------------------------------------------------------------------- steps --
class Case:
    """One request, alone in its call (chunks, from 17 tokens on)."""

    def __init__(self, T, H, P, N, rate, step, seed, scale=1.0):
        x, b, c = (synth.normal_bf16((T, h, n), seed + i, device="cuda")
                   for i, (h, n) in enumerate(((H, P), (1, N), (1, N))))
        self.ins = [x, step, b * scale, c]
        self.w = phs.ScanWeights(torch.full((H,), rate, device="cuda"))
        self.pool = phs.ScanPool.zeros(1, H, P, N)

    def check(self, chunked=True):
        T = self.ins[0].shape[0]
        out = phs.selective_scan_prompt(*self.ins, dev([0, T]), T, self.pool, self.w)
        y, S, m, A, log = ref.scan(*self.ins, torch.zeros_like(self.pool.s[0]), self.w.rate, None, None)
        bo, bs = ref.scan_bounds(y, m, A, log, out.dtype, self.ins[2].shape[2], chunked)
        # (fp32's lowest normal number is 2^-126: what is below may go out as zero, and
        # comes in again times up to N values of c below 2^3)
        ref.close(out, y, bo + 2.0 ** -115, "out")
        ref.close(self.pool.s[0], S, bs + 2.0 ** -120, "state")


@pytest.mark.parametrize("at,first", [(0, 1), (32, 33), (96, 104)])
@pytest.mark.parametrize("dt", [-35.0, -41.0, -60.0])
def test_a_tiny_step_before_a_strong_decay(at, first, dt):
    """A step of 2^-50 to 2^-87 whose 32 tokens decay by up to 2^-99 behind it:
    its own row is that step times c b x, and nothing else is in it."""
    step = torch.full((128, 2), -100.0, device="cuda")
    step[at] = dt
    step[first:at + 16] = 4.5    # softplus: 4.511
    Case(128, 2, 64, 64, -0.98, step, 5).check()


@pytest.mark.parametrize("big", [2.0 ** 30, 2.0 ** 40, 2.0 ** 60])
def test_huge_steps_that_decay_strongly(big):
    """Steps far above softplus's bend, each decaying by 2^-6 (32 tokens by
    2^-186): a weight is a step at most, whatever the factors it is formed of."""
    step = torch.full((300, 2), big, device="cuda")
    Case(300, 2, 64, 64, -4.15 / big, step, 7, 2.0 ** -20).check()


@pytest.mark.parametrize("B,lens,H,P,N", [
    (16, [4] * 16, 8, 64, 128),                     # token by token
    (1, [3000], 4, 64, 128),                        # cut into segments
    (2, [700, 40], 3, 128, 64), (40, [130] * 40, 16, 64, 64)])
def test_nothing_is_written_behind_the_workspace(B, lens, H, P, N):
    """A workspace of the very size, full of NaN as a call may find it."""
    cu = np.concatenate([[0], np.cumsum(lens)])
    T = int(cu[-1])
    x, b, c = (synth.normal_bf16((T, h, n), i, device="cuda")
               for i, (h, n) in enumerate(((H, P), (1, N), (1, N))))
    dt = synth.normal_bf16((T, H), 9, device="cuda")
    w = phs.ScanWeights(torch.full((H,), -2.0, device="cuda"))
    need = phs.scan_prompt_workspace_bytes(B, H, 1, P, N, T, max(lens))
    ws = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    outs = []
    for memory in (None, ws[:need]):
        pool = phs.ScanPool.zeros(B, H, P, N)
        outs += [phs.selective_scan_prompt(x, dt, b, c, dev(cu), max(lens), pool, w, workspace=memory),
                 pool.s]
    assert bool((ws[need:] == 0xFF).all())
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3])
    if need > 256:
        with pytest.raises(phs.PhsError):
            phs.selective_scan_prompt(x, dt, b, c, dev(cu), max(lens), pool, w, workspace=ws[:need - 256])


# ---------------------------------------------------- order of the requests --
# Calls with more (request, pair of heads) than SMs take the longest requests
# first, up to 256 requests.  Lengths of up to three chunks are never cut into
# segments, so that a request alone gives the same bits.
def alone(ins, lo, hi, start, resume, w):
    pool = phs.ScanPool(start.clone()[None])
    out = phs.selective_scan_prompt(*(t[lo:hi] for t in ins), dev([0, hi - lo]), hi - lo, pool, w,
                                    resume=dev([resume]))
    return out, pool.s[0]


def batch_of(lens, H, P, N, seed):
    T, B = int(sum(lens)), len(lens)
    x, b, c = (synth.normal_bf16((T, h, n), seed + i, device="cuda")
               for i, (h, n) in enumerate(((H, P), (1, N), (1, N))))
    dt = synth.normal_bf16((T, H), seed + 3, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = phs.ScanWeights(-1 - 15 * torch.rand(H, generator=g, device="cuda"),
                        torch.randn(H, generator=g, device="cuda"),
                        torch.randn(H, generator=g, device="cuda") - 3)
    start = torch.randn((B, H, P, N), generator=g, device="cuda")
    return [x, dt, b, c], w, start


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


MIXED = [0, 17, 300, 300, 16, 129, 128, 127, 1, 300, 256, 257, 40, 0, 384, 15]
ORDERS = {
    "mixed": MIXED * 4, "equal": [130] * 64, "one long": [3] * 40 + [384] + [16] * 23,
    "falling": list(range(320, 0, -5)), "rising": list(range(5, 325, 5)),
    "none long": [16, 0, 1, 8] * 16, "all long": [20 + 7 * (i * 29 % 50) for i in range(64)],
    "256": [17 + i * 37 % 150 for i in range(256)], "257": [17 + i * 37 % 150 for i in range(257)],
}


@pytest.mark.parametrize("P,N", [(64, 64), (128, 128)])
@pytest.mark.parametrize("name", ORDERS)
def test_every_request_of_a_full_call_is_taken_once(name, P, N):
    lens, H = ORDERS[name], 16
    B = len(lens)
    assert B * H * (P // 64) // 2 > sms()
    ins, w, start = batch_of(lens, H, P, N, B)
    cu = np.concatenate([[0], np.cumsum(lens)])
    rng = np.random.default_rng(B)
    ids, resume = rng.permutation(B), rng.integers(0, 2, B)
    ids[5] = -3
    runs = []
    for _ in range(2):   # (the same bits each time)
        pool, st = phs.ScanPool(start.clone()), torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full(ins[0].shape, 2.0, dtype=torch.bfloat16, device="cuda")
        phs.selective_scan_prompt(*ins, dev(cu), max(lens), pool, w, state_ids=dev(ids),
                                  resume=dev(resume), out=out, status=st)
        assert int(st.item()) == 0
        runs.append((out, pool.s))
    assert torch.equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][1], runs[1][1])
    out, S = runs[0]
    for r in range(B):
        lo, hi = int(cu[r]), int(cu[r + 1])
        if ids[r] < 0:
            assert not out[lo:hi].any()
            continue
        y, s = alone(ins, lo, hi, start[ids[r]], int(resume[r]), w)
        assert torch.equal(out[lo:hi], y) and torch.equal(S[ids[r]], s), (r, lens[r])
    kept = [i for i in range(B) if i not in set(ids.tolist())]
    assert torch.equal(S[kept], start[kept])


@pytest.mark.parametrize("P,N", [(64, 128), (128, 64)])
def test_bad_requests_of_a_full_call(P, N):
    """Ranges that fall, begin before an earlier end or are too long, ids that
    others have or that lie outside the pool, among 64 requests by length."""
    H, B = 16, 64
    lens = [20 + 13 * (i * 29 % 20) for i in range(B)]
    ins, w, start = batch_of(lens, H, P, N, 3)
    cu = np.concatenate([[0], np.cumsum(lens)])
    T = int(cu[-1])
    cu[20] = cu[19] - 30         # 19 falls, 20 begins inside 18
    cu[41] = cu[40] + max(lens) + 9   # 40 is too long, the next ones begin inside it
    cu[50] = T + 5               # 49 ends behind the tokens, 50 begins there and falls
    most = max(lens)
    ids = np.arange(B)
    ids[7], ids[30], ids[33] = ids[3], B + 4, -1
    bad = {19, 20, 49, 50, 7, 30, 33}
    bad |= {b for b in range(B) if not 0 <= cu[b + 1] - cu[b] <= most}   # (41 falls too)
    bad |= {b for b in range(B) if any(cu[j] > cu[b] for j in range(b))}
    assert len(bad) < B - 5 and any(cu[b + 1] - cu[b] > most for b in bad)
    pool, st = phs.ScanPool(start.clone()), torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full(ins[0].shape, 2.0, dtype=torch.bfloat16, device="cuda")
    phs.selective_scan_prompt(*ins, dev(cu), most, pool, w, state_ids=dev(ids), out=out, status=st)
    assert int(st.item()) in (-1, -3)
    for r in range(B):
        if r in bad:
            if r != 7:
                assert ids[r] < 0 or ids[r] >= B or torch.equal(pool.s[r], start[r]), r
            continue
        y, s = alone(ins, int(cu[r]), int(cu[r + 1]), start[r], 0, w)
        assert torch.equal(out[cu[r]:cu[r + 1]], y) and torch.equal(pool.s[ids[r]], s), r
    assert torch.equal(pool.s[[7, 30, 33]], start[[7, 30, 33]])


# ------------------------------------------------------- what each token weighs --
# Bounds of single terms.  A relative rounding error is 2^-24 in fp32, 2^-8 in bf16.
def one_hot_rows(values, width, first=0):
    """[len(values), width]: values[i] in column (first + i) % width."""
    m = torch.zeros((len(values), width), dtype=values.dtype, device="cuda")
    i = torch.arange(len(values), device="cuda")
    m[i, (first + i) % width] = values
    return m


def bf16_of(x):
    return x.bfloat16().double()


@pytest.mark.parametrize("rate", [0.0, -1e-3])
@pytest.mark.parametrize("T,H,P,N", [(128, 2, 64, 128), (100, 1, 64, 128), (17, 2, 128, 64),
                                     (64, 3, 64, 64), (128, 1, 128, 128)])
def test_a_state_keeps_24_bits_of_each_token(T, H, P, N, rate):
    """Token t alone has a value in column t of b, so that each element of the
    state is one token's weight x b.  Its weight and its product with x round
    by 2^-24 each, three bf16 terms hold that to 2^-24, each of their three
    products loses up to 2^-23 of the running sum: 2^-21 in all and 2^-24 for
    the weight.  A decay's logarithm is off by 17 roundings of 2^-24 of the sum
    behind the token, its exponential by 2 ulp (2^-22).  Two bf16 terms leave
    up to 2^-16, which this must see."""
    assert T <= N
    x = synth.normal_bf16((T, H, P), 3, device="cuda")
    b = one_hot_rows(synth.normal_bf16((T,), 4, device="cuda"), N)[:, None]
    dt = torch.rand((T, H), generator=torch.Generator(device="cuda").manual_seed(T), device="cuda") * 19 + 21
    pool, w = phs.ScanPool.zeros(1, H, P, N), phs.ScanWeights(torch.full((H,), rate, device="cuda"))
    phs.selective_scan_prompt(x, dt, b, torch.zeros_like(b), dev([0, T]), T, pool, w)
    log = (dt.double() * w.rate.double()).abs()        # (softplus above 20 is its argument)
    behind = log.sum(0) - torch.cumsum(log, 0)
    weight = torch.exp(-behind) * dt.double()
    xw = weight[..., None] * x.double()                # [T, H, P]
    want = torch.einsum("thp,tn->hpn", xw, b[:, 0].double())
    rel = 2.0 ** -21 + 2.0 ** -24 + 17 * 2.0 ** -24 * behind + (2.0 ** -22 if rate else 0.0)
    bound = torch.einsum("thp,tn->hpn", xw.abs() * rel[..., None], b[:, 0].double().abs())
    ref.close(pool.s[0], want, bound, "state")
    hi = bf16_of(xw)
    two = torch.einsum("thp,tn->hpn", hi + bf16_of(xw - hi), b[:, 0].double())
    assert bool(((two - want).abs() > bound).any())


@pytest.mark.parametrize("H,P,N", [(2, 64, 128), (1, 128, 64)])
def test_a_long_prompt_keeps_24_bits_of_each_token(H, P, N):
    """The same for tokens spread over a prompt that goes in segments."""
    T = 23 * 128 + 40
    at = torch.arange(N, device="cuda") * (T // N) + 5
    x, dt = synth.normal_bf16((T, H, P), 3, device="cuda"), torch.full((T, H), 25.3, device="cuda")
    b = torch.zeros((T, 1, N), dtype=torch.bfloat16, device="cuda")
    b[at, 0] = one_hot_rows(synth.normal_bf16((N,), 4, device="cuda"), N)
    pool, w = phs.ScanPool.zeros(1, H, P, N), phs.ScanWeights(torch.zeros(H, device="cuda"))
    phs.selective_scan_prompt(x, dt, b, torch.zeros_like(b), dev([0, T]), T, pool, w)
    want = torch.einsum("thp,tn->hpn", x.double() * dt.double()[..., None], b[:, 0].double())
    ref.close(pool.s[0], want, want.abs() * 2.0 ** -21, "state")


@pytest.mark.parametrize("rate,lo,hi", [(-1.0, 1e-3, 0.1), (-8.0, 1e-3, 1.0), (0.0, 0.5, 0.5),
                                        (-0.5, 0.01, 20.0)])
@pytest.mark.parametrize("T,H,P,N", [(128, 1, 128, 64), (300, 1, 128, 128), (300, 2, 64, 128),
                                     (100, 1, 64, 64), (17, 2, 64, 64), (257, 3, 64, 128)])
@pytest.mark.parametrize("half", [0, 1])
def test_each_weight_of_a_prompts_rows(T, H, P, N, rate, lo, hi, half):
    """Token j alone has a value (1) in column j of x, so that column j of a row
    is what that token weighs in it: of a chunk's own tokens one bf16 rounding
    (2^-8), of earlier ones' state another for the row's own; 0 of later ones.
    The decay's logarithm is off by 2^-19 of the chunk's sum for each chunk
    (see scan_bounds), exponentials, steps and products by 2^-19."""
    first = half * P if P < T else 0   # the tokens with values
    g = torch.Generator(device="cuda").manual_seed(T)
    s = torch.rand((T, H), generator=g, device="cuda") * (hi - lo) + lo
    dt = torch.where(s > 20, s, torch.log(torch.expm1(s)))
    beta, gamma = (synth.normal_bf16((T,), i, device="cuda") for i in (4, 5))
    b, c = (torch.zeros((T, 1, N), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    b[:, 0, 7], c[:, 0, 7] = beta, gamma
    n = min(P, T - first)
    x = torch.zeros((T, H, P), dtype=torch.bfloat16, device="cuda")
    x[first:first + n] = one_hot_rows(torch.ones(n, dtype=torch.bfloat16, device="cuda"), P)[:, None]
    pool, w = phs.ScanPool.zeros(1, H, P, N), phs.ScanWeights(torch.full((H,), rate, device="cuda"))
    out = phs.selective_scan_prompt(x, dt, b, c, dev([0, T]), T, pool, w)
    y, S, m, A, log = ref.scan(x, dt, b, c, torch.zeros_like(pool.s[0]), w.rate, None, None)
    X = max(float(log[i:i + 128].abs().sum(0).max()) for i in range(0, T, 128))
    rel = torch.full((T, 1, 1), 2.0 ** -8, dtype=torch.float64, device="cuda")
    rel[128:] = 2 * 2.0 ** -8 + 2.0 ** -16
    # (a token of the same chunk as the row's: one rounding, in any chunk)
    rel = rel + 2.0 ** -19 * (1 + (T // 128 + 1) * X)
    ref.close(out, y, y.abs() * rel + 2.0 ** -115, "weights")


@pytest.mark.parametrize("silu,skip", [(False, 0.0), (False, 1.0), (True, 0.0), (True, 1.0)])
@pytest.mark.parametrize("H,P,N", [(2, 64, 128), (1, 128, 64)])
def test_the_rows_mean_error(H, P, N, silu, skip):
    """Root mean square error of a prompt's rows against that of rounding the
    exact rows to bf16.  Each weight and each element of the state before a
    chunk rounds as the row does, by up to 2^-8 of itself, independently: for
    terms without a common sign the squares of their errors add up to what the
    row's own rounding adds, terms with one cancel less.  A rounding's mean
    square is 2^-16 / 3 E[1 / m^2] of the square, m the value's mantissa: E is
    0.54 for one spread evenly over its logarithm, 0.45 to 0.6 for sums.  So at
    most sqrt(1 + 0.6 / 0.45) = 1.53."""
    T = 1500
    g = torch.Generator(device="cuda").manual_seed(P)
    x, b, c = (torch.randn((T, h, n), generator=g, device="cuda").bfloat16()
               for h, n in ((H, P), (1, N), (1, N)))
    if silu:
        x, b, c = (torch.nn.functional.silu(t) for t in (x, b, c))
    dt = torch.randn((T, H), generator=g, device="cuda") * 0.7
    w = phs.ScanWeights(torch.full((H,), -4.0, device="cuda"), torch.full((H,), skip, device="cuda"),
                        torch.full((H,), -4.0, device="cuda"))
    pool = phs.ScanPool.zeros(1, H, P, N)
    out = phs.selective_scan_prompt(x, dt, b, c, dev([0, T]), T, pool, w)
    y, *_ = ref.scan(x, dt, b, c, torch.zeros_like(pool.s[0]), w.rate, w.skip, w.dt_bias)
    rms = [float(((t.double() - y) ** 2).mean().sqrt()) for t in (out, y.bfloat16())]
    print(f"rows' error {rms[0]:.3e}, of their rounding {rms[1]:.3e}: {rms[0] / rms[1]:.3f}")
    assert rms[0] <= 1.53 * rms[1]


# -------------------------------------------------------------------- limits --
def test_as_many_requests_as_a_call_takes():
    """65,535 requests of 17 tokens (the first to go in chunks): each its own."""
    B, n, H, P, N = 65535, 17, 1, 64, 64
    ins, w, start = batch_of([n], H, P, N, 2)
    T = B * n
    ins = [torch.cat([t.expand(512, *t.shape).flatten(0, 1) * (0.5 + i / 256) for i in range(128)])
           [:T].contiguous() for t in (ins[0],)] + [t.repeat(B, *([1] * (t.dim() - 1))) for t in ins[1:]]
    cu = torch.arange(0, T + 1, n, dtype=torch.int32, device="cuda")
    pool, st = phs.ScanPool.zeros(B, H, P, N), torch.zeros(1, dtype=torch.int32, device="cuda")
    out = phs.selective_scan_prompt(*ins, cu, n, pool, w, status=st)
    assert int(st.item()) == 0
    for b in [*range(0, B, 509), 512 * 3 - 1, 512 * 3, B - 1]:
        y, s = alone(ins, b * n, b * n + n, torch.zeros_like(start[0]), 0, w)
        assert torch.equal(out[b * n:b * n + n], y) and torch.equal(pool.s[b], s), b


@pytest.mark.parametrize("H,G", [(65535, 1), (65534, 2)])
def test_as_many_heads_as_a_call_takes(H, G):
    T, P, N = 40, 64, 64
    x = synth.normal_bf16((T, 64, P), 1, device="cuda")
    x = torch.cat([x * (0.5 + i / 1024) for i in range(1024)], 1)[:, :H].contiguous()
    b, c = (synth.normal_bf16((T, G, N), i, device="cuda") for i in (2, 3))
    dt = synth.normal_bf16((T, 64), 4, device="cuda").repeat(1, 1024)[:, :H].contiguous()
    w = phs.ScanWeights(-1 - torch.arange(H, device="cuda") % 7 * 1.0)
    pool, st = phs.ScanPool.zeros(1, H, P, N), torch.zeros(1, dtype=torch.int32, device="cuda")
    out = phs.selective_scan_prompt(x, dt, b, c, dev([0, T]), T, pool, w, status=st)
    assert int(st.item()) == 0
    for h in (0, 1, 2, 4095, 32766, 32767, 32768, 65000, H - 2, H - 1):
        g, one = h // (H // G), phs.ScanPool.zeros(1, 1, P, N)
        y = phs.selective_scan_prompt(x[:, h:h + 1].contiguous(), dt[:, h:h + 1], b[:, g:g + 1],
                                      c[:, g:g + 1], dev([0, T]), T, one,
                                      phs.ScanWeights(w.rate[h:h + 1].contiguous()))
        assert torch.equal(out[:, h], y[:, 0]) and torch.equal(pool.s[0, h], one.s[0, 0]), h


@pytest.mark.parametrize("H,P,N", [(2, 64, 128), (3, 128, 64)])
@pytest.mark.parametrize("n", [0, 1, 16, 17, 129, 1000, 5990])
@pytest.mark.parametrize("resume", [0, 1])
def test_a_prompt_far_below_the_stated_length(H, P, N, n, resume):
    """The plan is made for 6,000 tokens, cut into segments; most of them then
    have no chunk."""
    L = Layer(H, 1, P, N, 2, H)
    ins = L.inputs(6000, 3)
    out, st = torch.full((6000, H, P), 2.0, dtype=torch.bfloat16, device="cuda"), \
        torch.zeros(1, dtype=torch.int32, device="cuda")
    phs.selective_scan_prompt(*ins, dev([3, 3 + n]), 6000, L.pool, L.w, state_ids=dev([1]),
                              resume=dev([resume]), out=out, status=st)
    assert int(st.item()) == 0
    L.check(ins, out, [(3, 3 + n)], [1], [resume], True)
    assert bool((out[:3] == 2).all()) and bool((out[3 + n:] == 2).all())


def test_a_captured_call_with_other_lengths_each_time():
    """Offsets, ids and resume are read on the device: a graph made for the
    longest call is replayed for others."""
    L = Layer(4, 2, 64, 128, 5, 7)
    ins = L.inputs(2000, 3)
    out = torch.zeros((2000, 4, 64), dtype=torch.bfloat16, device="cuda")
    cu, ids, resume = dev([0, 1000, 2000, 2000]), dev([0, 1, 2]), dev([0, 0, 0])
    need = phs.scan_prompt_workspace_bytes(3, 4, 2, 64, 128, 2000, 2000)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    call = lambda: phs.selective_scan_prompt(*ins, cu, 2000, L.pool, L.w, state_ids=ids, resume=resume,
                                             out=out, workspace=ws)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for offsets, i, r in (([0, 5, 1700, 1716], [4, 2, 0], [1, 0, 1]), ([0, 0, 2000, 2000], [3, 1, 2], [1, 1, 0]),
                          ([100, 117, 134, 151], [2, -1, 3], [0, 1, 1]), ([0, 700, 1400, 2000], [1, 0, 4], [1, 1, 1])):
        L.pool.s.copy_(L.start)
        out.fill_(2)
        cu.copy_(dev(offsets)), ids.copy_(dev(i)), resume.copy_(dev(r))
        ws.fill_(0xFF)
        graph.replay()
        L.check(ins, out, list(zip(offsets[:-1], offsets[1:])), i, r, True)
        assert bool((out[:offsets[0]] == 2).all()) and bool((out[offsets[-1]:] == 2).all())
