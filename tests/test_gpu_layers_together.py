"""Rotary cache writes, the convolution and the scan as a hybrid stack runs
them: prompts in parts, then tokens, through an attention layer whose cache is
partly held in 8 bits and a selective layer; captured and replayed; on other
streams."""
import math

import numpy as np
import pytest
import torch

import layers_ref as ref
import paged_hybrid_sliding_gb300 as phs
import synth
from gpu_util import ATOL, RTOL, dev

pytestmark = pytest.mark.gpu

D, HQ, HK = 64, 4, 2                    # attention
H, G, P, N, W = 4, 2, 64, 64, 4         # selective layer
C = H * P + 2 * G * N                   # its convolved channels
QKV, PROJ = (HQ + 2 * HK) * D, C + 8    # rows of the two projections, H of the last 8 steps
HOT = 20                                # tokens that stay in bf16


class Stack:
    def __init__(self, rows, most, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g, device="cuda")
        self.rope = phs.Rope.make(D, scaling="parts", scale=4.0, trained_len=64)
        self.freq, self.factor = phs.rope_frequencies(D, scaling="parts", scale=4.0, trained_len=64)
        self.conv = phs.ConvWeights(r(C, W) * 0.5, r(C) * 0.1)
        self.scan = phs.ScanWeights(-torch.rand(H, generator=g, device="cuda") * 4 - 0.5, r(H),
                                    r(H) - 2)
        self.table, pages = synth.block_tables_from_permutation(
            synth.pages_needed(np.full(rows, most)), seed)
        self.qtable, qpages = synth.block_tables_from_permutation(np.full(rows, most // 32), seed + 1)
        self.pool = phs.PagedPool.empty(pages, HK, D)
        self.int8 = phs.Int8Pool.empty(qpages, HK, D)
        self.inputs = phs.ConvPool(r(rows, W - 1, C).bfloat16())
        self.states = phs.ScanPool(r(rows, H, P, N))
        self.lens = np.zeros(rows, np.int32)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def selective(self, rows, cu, ids, resume):
        """Prompts (cu given) or one token each through the selective layer."""
        x = rows[:, :C]
        if cu is None:
            y = phs.causal_conv_decode(x, self.inputs, self.conv, state_ids=ids, status=self.status)
        else:
            y = phs.causal_conv_prompt(x, cu, self.inputs, self.conv, state_ids=ids, resume=resume,
                                       status=self.status)
        x, b, c = y.split([H * P, G * N, G * N], 1)
        a = (x.unflatten(1, (H, P)), rows[:, C:C + H], b.unflatten(1, (G, N)), c.unflatten(1, (G, N)))
        if cu is None:
            return phs.selective_scan_decode(*a, self.states, self.scan, state_ids=ids,
                                             out_dtype=torch.float32, status=self.status)
        return phs.selective_scan_prompt(*a, cu, 200, self.states, self.scan, state_ids=ids,
                                         resume=resume, status=self.status)

    def write(self, rows, cu, before, lens):
        """Rotate and write the rows' keys and values, the old ones in 8 bits."""
        t = rows.shape[0]
        q, k, v = (x.unflatten(1, (-1, D)) for x in rows.split([HQ * D, HK * D, HK * D], 1))
        was, now = (np.maximum(n - HOT, 0) // 32 * 32 for n in (before, lens))
        most = int((now - was).max()) // 32
        return phs.kv_write_paged(self.pool, k, v, dev(self.table), dev(lens), cu_seqlens=cu, q=q,
                                  rope=self.rope, int8=self.int8, qtable=dev(self.qtable),
                                  qlens_before=dev(was), qlens=dev(now), max_qblocks=most,
                                  status=self.status), dev(now)

    def attend(self, q, lens, qlens):
        return phs.attn_decode_full_paged(q, self.pool, dev(self.table), dev(lens), 256,
                                          int8=self.int8, qtable=dev(self.qtable), qlens=qlens,
                                          out_dtype=torch.float32, status=self.status)


def test_prompts_in_parts_then_tokens():
    rows = 3
    s = Stack(rows, 256, 5)
    start = s.inputs.c.clone(), s.states.s.clone()
    parts = [[70, 33, 1], [1, 150, 40], [0, 3, 64]]
    kv, proj, outs = ([[] for _ in range(rows)] for _ in range(3))   # histories
    ids = np.array([2, 0, 1], np.int32)
    for i, part in enumerate(parts):
        cu = dev(np.concatenate([[0], np.cumsum(part)]))
        t = sum(part)
        qkv = synth.normal_bf16((t, QKV), 100 + i, device="cuda")
        pr = synth.normal_bf16((t, PROJ), 200 + i, device="cuda")
        before, lens = s.lens.copy(), s.lens + np.array(part, np.int32)
        s.write(qkv, cu, before, lens)
        y = s.selective(pr, cu, dev(ids), dev([i > 0] * rows))
        s.lens = lens
        at = 0
        for b, n in enumerate(part):
            kv[b].append(qkv[at:at + n])
            proj[b].append(pr[at:at + n])
            outs[b].append(y[at:at + n].float())
            at += n
    for step in range(6):
        qkv = synth.normal_bf16((rows, QKV), 300 + step, device="cuda")
        pr = synth.normal_bf16((rows, PROJ), 400 + step, device="cuda")
        before, lens = s.lens.copy(), s.lens + 1
        q, qlens = s.write(qkv, None, before, lens)
        o = s.attend(q, lens, qlens)
        y = s.selective(pr, None, dev(ids), None)
        s.lens = lens
        for b in range(rows):
            kv[b].append(qkv[b:b + 1])
            proj[b].append(pr[b:b + 1])
            outs[b].append(y[b:b + 1])
    assert int(s.status.item()) == 0
    # attention of the last token over the cache as it reads back, and the cache
    # against what was written
    cu = np.concatenate([[0], np.cumsum(s.lens)])
    ko, vo = phs.kv_read_paged(s.pool, dev(s.table), dev([0] * rows), dev(cu), int(cu[-1]), 256,
                               int8=s.int8, qtable=dev(s.qtable), qlens=qlens, status=s.status)
    for b in range(rows):
        n, k, v = int(s.lens[b]), ko[cu[b]:cu[b + 1]].double(), vo[cu[b]:cu[b + 1]].double()
        rows_b = torch.cat(kv[b])
        kr, e = ref.rotated(rows_b[:, HQ * D:(HQ + HK) * D].unflatten(1, (HK, D)),
                            torch.arange(n, device="cuda"), s.freq, False, s.factor)
        old = max(n - HOT, 0) // 32 * 32
        # half a code's step of a block's absmax, and twice bf16's
        step = kr.abs().amax() / 127 / 2
        err = (k - kr).abs() - e - kr.abs() * 2.0 ** -8
        assert bool((err[old:] <= 0).all()) and bool((err[:old] <= step * 1.01).all())
        for h in range(HQ):
            p = torch.softmax(k[:, h // 2] @ q[b, h].double() / math.sqrt(D), 0)
            want = p @ v[:, h // 2]
            assert bool(((o[b, h].double() - want).abs() <= ATOL + RTOL * want.abs()).all())
        # the selective layer from its first token
        x = torch.cat(proj[b])
        zero = torch.zeros_like(start[0][0])
        y, e, last = ref.conv(x[:, :C], zero, s.conv.weight, s.conv.bias, True)
        assert torch.equal(s.inputs.c[ids[b]], last)
        # (the scan reads the convolution's bf16 rows)
        y = phs.causal_conv_prompt(x[:, :C], dev([0, n]), phs.ConvPool.zeros(1, C, W), s.conv)
        xs, bs, cs = y.split([H * P, G * N, G * N], 1)
        want, S, m, A, log = ref.scan(xs.unflatten(1, (H, P)), x[:, C:C + H], bs.unflatten(1, (G, N)),
                                      cs.unflatten(1, (G, N)), torch.zeros_like(start[1][0]),
                                      s.scan.rate, s.scan.skip, s.scan.dt_bias)
        bo, bs = ref.scan_bounds(want, m, A, log, torch.bfloat16, N, True)
        ref.close(torch.cat(outs[b]), want, bo, f"scan {b}")
        ref.close(s.states.s[ids[b]], S, bs, f"state {b}")


def test_a_captured_step_is_the_eager_one():
    """A token through both layers, replayed: bit for bit the eager calls."""
    rows = 3
    runs = []
    for captured in (False, True):
        s = Stack(rows, 64, 7)
        s.pool.k.zero_(), s.pool.v.zero_()
        qkv = synth.normal_bf16((rows, QKV), 1, device="cuda")
        pr = synth.normal_bf16((rows, PROJ), 2, device="cuda")
        ids, lens, table, zero = dev([0, 1, 2]), dev([5, 17, 40]), dev(s.table), dev([0, 0, 0])
        qt, q32 = dev(s.qtable), dev([0, 0, 32])

        def step():
            q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([HQ * D, HK * D, HK * D], 1))
            q = phs.kv_write_paged(s.pool, k, v, table, lens, q=q, rope=s.rope, int8=s.int8,
                                   qtable=qt, qlens_before=zero, qlens=q32, max_qblocks=1)
            o = phs.attn_decode_full_paged(q, s.pool, table, lens, 64, int8=s.int8, qtable=qt,
                                           qlens=q32)
            return q, o, s.selective(pr, None, ids, None)

        if captured:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                step()
            torch.cuda.current_stream().wait_stream(side)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                outs = step()
            graph.replay()
            graph.replay()
        else:
            for _ in range(3):
                outs = step()
        torch.cuda.synchronize()
        runs.append([*outs, s.pool.k, s.pool.v, s.int8.k[s.qtable[2][0]], s.int8.v[s.qtable[2][0]],
                     s.inputs.c, s.states.s])
    for a, b in zip(*runs):
        assert torch.equal(a, b)


def scan_inputs(T, heads, groups, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    mk = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    w = phs.ScanWeights(-torch.rand(heads, generator=g, device="cuda") - 0.1)
    return (mk(T, heads, 64), mk(T, heads), mk(T, groups, 128), mk(T, groups, 128)), w


def test_two_graphs_with_their_own_workspaces_replayed_at_once():
    T, heads = 1500, 4
    pool = phs.ScanPool.zeros(2, heads, 64, 128)
    need = phs.scan_prompt_workspace_bytes(1, heads, 2, 64, 128, T, T)
    runs = []
    for r in range(2):
        ins, w = scan_inputs(T, heads, 2, r)
        args = dict(state_ids=dev([r]), resume=dev([1]), out=torch.empty_like(ins[0]),
                    workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
        cu = dev([0, T])
        phs.selective_scan_prompt(*ins, cu, T, pool, w, **args)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            phs.selective_scan_prompt(*ins, cu, T, pool, w, **args)
        runs.append((graph, args["out"], (ins, w, cu, args)))
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
        for st, (graph, _, _) in zip(streams, runs):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for a, (_, out, _) in zip(want, runs):
        assert torch.equal(a, out)
    assert torch.equal(states, pool.s)


def test_memory_of_a_call_on_another_stream():
    """What the current stream has let go of, but is still to write, is not
    what a call on another stream gets for its output and workspace."""
    T, heads = 1200, 4
    ins, w = scan_inputs(T, heads, 1, 3)
    cu = dev([0, T])
    need = phs.scan_prompt_workspace_bytes(1, heads, 1, 64, 128, T, T)
    want = phs.selective_scan_prompt(*ins, cu, T, phs.ScanPool.zeros(1, heads, 64, 128), w)
    side = torch.cuda.Stream()
    pool = phs.ScanPool.zeros(1, heads, 64, 128)
    torch.cuda.synchronize()
    # (sleeps about 20 ms, far longer than the call)
    waste = [torch.empty(n, dtype=torch.uint8, device="cuda")
             for n in (need, want.numel() * 2) for _ in range(4)]
    torch.cuda._sleep(40_000_000)
    for x in waste:
        x.fill_(255)
    del waste, x
    got = phs.selective_scan_prompt(*ins, cu, T, pool, w, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_calls_are_the_same_every_time():
    """No order of atomics or of CTAs in any result."""
    s, t = Stack(3, 256, 9), Stack(3, 256, 9)
    qkv = synth.normal_bf16((300, QKV), 1, device="cuda")
    pr = synth.normal_bf16((300, PROJ), 2, device="cuda")
    cu, ids = dev([0, 199, 200, 300]), dev([0, 1, 2])
    lens = np.array([199, 1, 100], np.int32)
    got = []
    for x in (s, t):
        x.pool.k.zero_(), x.pool.v.zero_()
        for y in (x.int8.k, x.int8.v, x.int8.k_scale, x.int8.v_scale):
            y.zero_()
        q, _ = x.write(qkv, cu, np.zeros(3, np.int32), lens)
        y = x.selective(pr, cu, ids, dev([1, 0, 1]))
        got.append([q, y, x.pool.k, x.pool.v, x.int8.k, x.int8.v, x.inputs.c, x.states.s])
    for a, b in zip(*got):
        assert torch.equal(a, b)
