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
