"""The page operations, differential decode and linear attention as a server
of sampled continuations runs them: a prompt, children of it, tokens in each,
some of them dropped, the pool compacted, more tokens."""
import math

import numpy as np
import pytest
import torch

import ops_ref
import paged_hybrid_sliding_gb300 as phs
import synth
from gpu_util import dev

pytestmark = pytest.mark.gpu

D, H, HV = 64, 4, 2          # differential heads and value heads
LQ, LKV = 4, 2               # linear attention heads
ROWS, PAGES, WIDTH = 8, 64, 12


class Server:
    """Block table rows and states of the same numbers, one layer of each kind."""

    def __init__(self, seed):
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        kv = [self.bf16(PAGES, 2 * HV, 16, D) for _ in range(2)]
        self.pool = phs.PagedPool(*kv)
        self.table = torch.full((ROWS, WIDTH), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(ROWS, dtype=torch.int32, device="cuda")
        self.counts = torch.zeros(PAGES, dtype=torch.int32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.states = phs.StatePool.zeros(ROWS, LKV, D)
        self.decay = -torch.logspace(-3, -0.2, LKV, device="cuda")
        vec = lambda: torch.randn(D, generator=self.gen, device="cuda") * 0.1
        self.weights = phs.DiffWeights(vec(), vec(), vec(), vec(), 0.8,
                                       torch.rand(2 * D, generator=self.gen, device="cuda") + 0.5)
        self.history = [[] for _ in range(ROWS)]     # (diff k, v, linear k, v) of each token

    def bf16(self, *shape):
        return torch.randn(shape, generator=self.gen, device="cuda").to(torch.bfloat16)

    def prompt(self, row, n, alloc):
        pages = alloc.alloc((n + 15) // 16)
        self.table[row, :len(pages)] = dev(pages)
        self.counts.copy_(dev(alloc.refcounts().astype(np.int32)))
        k, v = self.bf16(n, 2 * HV, D), self.bf16(n, 2 * HV, D)
        for t in range(n):
            self.pool.k[pages[t // 16], :, t % 16] = k[t]
            self.pool.v[pages[t // 16], :, t % 16] = v[t]
        self.lens[row] = n
        q, lk, lv = self.bf16(n, LQ, D), self.bf16(n, LKV, D), self.bf16(n, LKV, D)
        out = phs.linear_attn_prompt(q, lk, lv, dev([0, n]), n, self.states, self.decay,
                                     state_ids=dev([row]), status=self.status)
        self.history[row] = [(k[t], v[t], lk[t], lv[t]) for t in range(n)]
        return q, out

    def fork(self, src, dst):
        phs.pages_fork([self.pool], self.table, self.lens, self.counts, dev(src), dev(dst),
                       status=self.status)
        self.states.s[dst] = self.states.s[src]
        for a, b in zip(src, dst):
            self.history[b] = list(self.history[a])

    def free(self, rows):
        phs.pages_free(self.table, self.lens, self.counts, dev(rows), status=self.status)
        for r in rows:
            self.history[r] = []

    def token(self, rows):
        """One token for each of `rows`, whose pages have room for it."""
        n = len(rows)
        k, v = self.bf16(n, 2 * HV, D), self.bf16(n, 2 * HV, D)
        q, lq = self.bf16(n, 2 * H, D), self.bf16(n, LQ, D)
        lk, lv = self.bf16(n, LKV, D), self.bf16(n, LKV, D)
        self.lens[rows] += 1
        out = phs.attn_decode_diff_paged(q, self.pool, self.table[rows], self.lens[rows],
                                         WIDTH * 16, self.weights, out_dtype=torch.float32,
                                         k_new=k, v_new=v, page_refcount=self.counts,
                                         status=self.status)
        lin = phs.linear_attn_decode(lq, lk, lv, self.states, self.decay, state_ids=dev(rows),
                                     out_dtype=torch.float32, status=self.status)
        for i, r in enumerate(rows):
            self.history[r].append((k[i], v[i], lk[i], lv[i]))
        return q, out, lq, lin

    def check(self, rows, q, out, lq, lin):
        assert int(self.status.item()) == 0
        for i, r in enumerate(rows):
            k, v, lk, lv = (torch.stack(x).double() for x in zip(*self.history[r]))
            n, used = len(lk), ops_ref.pages(len(lk))
            kv = [torch.cat([x, x.new_zeros((used * 16 - n, 2 * HV, D))])
                  .view(used, 16, 2 * HV, D).transpose(1, 2) for x in (k, v)]
            w = self.weights
            ref, bound = ops_ref.diff_decode(
                q[i:i + 1], *kv, np.arange(used, dtype=np.int32)[None], [n],
                (w.lambda_q1, w.lambda_k1, w.lambda_q2, w.lambda_k2), w.lambda_init,
                w.norm_weight, w.norm_eps, 1 / math.sqrt(D), 2.0**-24)
            assert bool(((out[i].double() - ref[0]).abs() <= bound[0]).all()), r
            keep = torch.exp(self.decay.double()[None] *
                             torch.arange(n - 1, -1, -1, device="cuda")[:, None])
            S = torch.einsum("nh,nhd,nhe->hde", keep, lk, lv)
            A = torch.einsum("nh,nhd,nhe->hde", keep, lk.abs(), lv.abs())
            qi = lq[i].double().view(LKV, LQ // LKV, D) / math.sqrt(D)
            ref = torch.einsum("hgd,hde->hge", qi, S).reshape(LQ, D)
            mag = torch.einsum("hgd,hde->hge", qi.abs(), A).reshape(LQ, D)
            # (n + 8 + D) roundings of 2^-22 at most, of the absolute sums
            assert bool(((lin[i].double() - ref).abs() <= mag * (n + 8 + D) * 2.0**-22).all()), r


@pytest.mark.parametrize("n", [1, 16, 37, 150])
def test_sampled_continuations(n):
    s, alloc = Server(n), phs.PageAllocator(PAGES)
    hold = alloc.alloc(5)                       # pages of another request, freed later
    q, out = s.prompt(0, n, alloc)
    assert torch.isfinite(out.float()).all()
    # room for the tokens to come in the first row's last page, or one more
    def room(rows):
        for r in rows:
            if int(s.lens[r]) % 16 == 0:
                page, = alloc_from_counts()
                s.table[r, int(s.lens[r]) // 16] = page
                s.counts[page] = 1

    def alloc_from_counts():
        alloc.load_refcounts(s.counts.cpu().numpy())
        page = alloc.alloc(1)
        return page

    rows = [0, 3, 5, 6]
    s.fork([0, 0, 0], [3, 5, 6])
    for _ in range(3):
        room(rows)
        s.check(rows, *s.token(rows))
    s.free([5, 0])
    rows = [6, 3]
    s.counts[hold] -= 1                         # a hole in front
    page_map, live = phs.pages_compact([s.pool], s.table, s.lens, s.counts, status=s.status)
    assert int(live.item()) == int((s.counts > 0).sum())
    assert not s.counts[int(live.item()):].any()
    for _ in range(2):
        room(rows)
        s.check(rows, *s.token(rows))
    # a grandchild in a freed row
    s.fork([3], [0])
    rows = [0, 3, 6]
    room(rows)
    s.check(rows, *s.token(rows))
    s.free([0, 3, 6])
    assert not s.counts.any() and not s.lens.any()


def test_decode_is_the_same_after_compaction():
    """Moving pages changes no bit of any output."""
    s, alloc = Server(3), phs.PageAllocator(PAGES)
    hold = alloc.alloc(7)
    s.prompt(2, 100, alloc)
    s.fork([2], [4])
    s.counts[hold] -= 1
    q = s.bf16(2, 2 * H, D)
    rows = torch.tensor([2, 4], device="cuda")

    def decode():
        return phs.attn_decode_diff_paged(q, s.pool, s.table[rows], s.lens[rows], 192, s.weights,
                                          out_dtype=torch.float32, status=s.status)

    before = decode()
    page_map, _ = phs.pages_compact([s.pool], s.table, s.lens, s.counts, status=s.status)
    assert (page_map.cpu().numpy() != np.arange(PAGES)).any()
    assert torch.equal(before, decode())
    assert int(s.status.item()) == 0


def test_two_graphs_with_their_own_workspaces_replayed_at_once():
    """Two captured steps on two streams: no state between them but the pool
    rows that each updates."""
    D, Hq, Hkv, T = 128, 16, 2, 1300
    gen = torch.Generator(device="cuda").manual_seed(8)
    mk = lambda *shape: torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)
    decay = -torch.logspace(-4, -0.5, Hkv, device="cuda")
    pool = phs.StatePool.zeros(2, Hkv, D)
    need = phs.linear_prompt_workspace_bytes(1, Hq, Hkv, D, T, T)
    runs = []
    for r in range(2):
        q, k, v = mk(T, Hq, D), mk(T, Hkv, D), mk(T, Hkv, D)
        args = dict(state_ids=dev([r]), resume=dev([1]), out=torch.empty_like(q),
                    workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
        cu = dev([0, T])
        phs.linear_attn_prompt(q, k, v, cu, T, pool, decay, **args)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            phs.linear_attn_prompt(q, k, v, cu, T, pool, decay, **args)
        runs.append((graph, args["out"], (q, k, v, cu, args)))
    pool.s.zero_()
    want = []
    for graph, out, _ in runs:
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        want.append(out.clone())
    states = pool.s.clone()
    pool.s.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(2):
        for s, (graph, _, _) in zip(streams, runs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for w, (_, out, _) in zip(want, runs):
        assert torch.equal(w, out)
    assert torch.equal(states, pool.s)


def test_memory_of_a_call_on_another_stream():
    """What the current stream has let go of, but is still to write, is not
    what a call on another stream gets for its output and workspace."""
    D, Hq, Hkv, T = 128, 4, 2, 1200
    gen = torch.Generator(device="cuda").manual_seed(9)
    mk = lambda *shape: torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)
    q, k, v = mk(T, Hq, D), mk(T, Hkv, D), mk(T, Hkv, D)
    decay = -torch.logspace(-4, -0.5, Hkv, device="cuda")
    cu = dev([0, T])
    need = phs.linear_prompt_workspace_bytes(1, Hq, Hkv, D, T, T)
    want = phs.linear_attn_prompt(q, k, v, cu, T, phs.StatePool.zeros(1, Hkv, D), decay)
    side = torch.cuda.Stream()
    pool = phs.StatePool.zeros(1, Hkv, D)
    torch.cuda.synchronize()
    # (sleeps about 20 ms, far longer than the call)
    waste = [torch.empty(n, dtype=torch.uint8, device="cuda")
             for n in (need, want.numel() * 2) for _ in range(4)]
    torch.cuda._sleep(40_000_000)
    for w in waste:
        w.fill_(255)
    del waste, w
    got = phs.linear_attn_prompt(q, k, v, cu, T, pool, decay, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
