"""Rotary positions, cache writes (bf16 pages and 8-bit blocks) and the cache
read back, against the definitions and the single-token calls."""
import numpy as np
import pytest
import torch

import layers_ref as ref
import paged_hybrid_sliding_gb300 as phs
import synth
from gpu_util import dev

pytestmark = pytest.mark.gpu


def bf16(shape, seed):
    return synth.normal_bf16(shape, seed, device="cuda")


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def strided(t, pad):
    """The same values as rows of a wider tensor."""
    w = torch.full((t.shape[0], t[0].numel() + pad), 7.0, dtype=t.dtype, device=t.device)
    w[:, pad:] = t.flatten(1)
    return w[:, pad:].unflatten(1, t.shape[1:])


ROPES = [(64, 64, False), (64, 64, True), (128, 128, False), (128, 128, True), (128, 64, False),
         (128, 64, True), (64, 16, False), (128, 16, True), (128, 48, False), (128, 48, True)]


@pytest.mark.parametrize("D,rotary,inter", ROPES)
@pytest.mark.parametrize("T,Hq,Hk", [(1, 1, 1), (2, 4, 2), (37, 32, 8), (300, 5, 5)])
def test_rotate(D, rotary, inter, T, Hq, Hk):
    rope = phs.Rope.make(rotary, interleaved=inter, scaling="wavelengths", scale=4.0,
                         trained_len=2048, factor=1.25)
    f = phs.rope_frequencies(rotary, scaling="wavelengths", scale=4.0, trained_len=2048)[0]
    q, k = strided(bf16((T, Hq, D), 1), 24), strided(bf16((T, Hk, D), 2), 8)
    pos = torch.randint(0, 300_000, (T,), dtype=torch.int32, device="cuda")
    pos[0] = 2**31 - 1
    qo, ko = phs.rope_rotate(q, k, pos, rope)
    for x, y in ((q, qo), (k, ko)):
        r, e = ref.rotated(x, pos, f, inter, 1.25)
        ref.close(y, r, e, "rotated")
    # without k, and in place
    assert torch.equal(phs.rope_rotate(q, None, pos, rope)[0], qo)
    q2, k2 = phs.rope_rotate(q, k, pos, rope, q_out=q, k_out=k)
    assert q2 is q and torch.equal(q, qo) and torch.equal(k, ko)


@pytest.mark.parametrize("T", [1, 3, 50])
def test_rotate_parts_of_one_projection(T):
    """q, k and v side by side in one row: q and k in place, or into parts of
    other rows; nothing else changes."""
    Hq, Hk, D = 4, 2, 64
    rope, pos = phs.Rope.make(D), torch.arange(5, 5 + T, dtype=torch.int32, device="cuda")
    rows = bf16((T, Hq + 2 * Hk, D), 4)
    want = phs.rope_rotate(rows[:, :Hq].contiguous(), rows[:, Hq:Hq + Hk].contiguous(), pos, rope)
    want = torch.cat([*want, rows[:, Hq + Hk:]], 1)
    into = rows.clone()
    parts = lambda r: (r[:, :Hq], r[:, Hq:Hq + Hk])
    phs.rope_rotate(*parts(rows), pos, rope, *parts(into))
    assert torch.equal(into, want)
    phs.rope_rotate(*parts(rows), pos, rope, *parts(rows))
    assert torch.equal(rows, want)
    # an output over a part of an input is refused
    before = rows.clone()
    with pytest.raises(RuntimeError):
        phs.rope_rotate(*parts(rows), pos, rope, rows[:, 1:1 + Hq], into[:, :Hk])
    assert torch.equal(rows, before)


def test_rotate_many_tokens():
    """Every tile size, and heads above one pass of a CTA."""
    rope = phs.Rope.make(64)
    f = phs.rope_frequencies(64)[0]
    q = bf16((10001, 17, 64), 3)
    pos = torch.arange(10001, dtype=torch.int32, device="cuda")
    whole, _ = phs.rope_rotate(q, None, pos, rope)
    r, e = ref.rotated(q[::97], pos[::97], f, False, 1.0)
    ref.close(whole[::97], r, e, "rotated")
    for lo, hi in ((0, 1), (5, 700), (100, 2000), (77, 4000)):
        part, _ = phs.rope_rotate(q[lo:hi], None, pos[lo:hi], rope)
        assert torch.equal(part, whole[lo:hi])


class Cache:
    """Pools and tables of requests of given lengths; unused table entries -1."""

    def __init__(self, lens, H, D, seed, spare=3, qlens=None, scatter=True):
        self.lens = np.asarray(lens, np.int32)
        self.table, n = synth.block_tables_from_permutation(
            synth.pages_needed(self.lens), seed, width=int(synth.pages_needed(self.lens).max()) + 1)
        self.pool = phs.PagedPool(bf16((n + spare, H, 16, D), seed + 1), bf16((n + spare, H, 16, D), seed + 2))
        self.start = phs.PagedPool(self.pool.k.clone(), self.pool.v.clone())
        if qlens is not None:
            self.qlens = np.asarray(qlens, np.int32)
            self.qtable, n = synth.block_tables_from_permutation(
                self.qlens // 32, seed + 3, width=int(self.qlens.max()) // 32 + 1)
            g = torch.Generator(device="cuda").manual_seed(seed)
            self.int8 = phs.Int8Pool.empty(n + spare, H, D)
            for t in (self.int8.k, self.int8.v):
                t.random_(1, 256, generator=g)
            for t in (self.int8.k_scale, self.int8.v_scale):
                t.uniform_(0.5, 1.5, generator=g)
            self.int8_start = phs.Int8Pool(*[t.clone() for t in (
                self.int8.k, self.int8.v, self.int8.k_scale, self.int8.v_scale)])

    def rows(self, pool_t, b, lo, hi):
        """Tokens [lo, hi) of request b, [tokens, H, D]."""
        t = np.arange(lo, hi)
        page = torch.from_numpy(self.table[b][t // 16].astype(np.int64)).cuda()
        return pool_t[page, :, torch.from_numpy(t % 16).cuda()]


def same(pool, other):
    return torch.equal(pool.k, other.k) and torch.equal(pool.v, other.v)


LENS = [[1], [0, 5, 0], [16, 17, 15, 32], [1, 100, 3, 257], [2000]]


@pytest.mark.parametrize("new", LENS)
@pytest.mark.parametrize("H,D", [(1, 64), (8, 128), (3, 128)])
def test_write_prompts(new, H, D):
    new = np.array(new, np.int32)
    old = np.array([(7 * i * i) % 40 for i in range(len(new))], np.int32)
    c = Cache(new + old, H, D, 11)
    T = int(new.sum())
    cu = np.concatenate([[0], np.cumsum(new)])
    k, v, q = strided(bf16((T, H, D), 1), 8), strided(bf16((T, H, D), 2), 16), bf16((T, 2 * H, D), 3)
    st = status()
    assert phs.kv_write_paged(c.pool, k, v, dev(c.table), dev(c.lens), cu_seqlens=dev(cu),
                              status=st) is None
    assert int(st.item()) == 0
    rope = phs.Rope.make(D)
    r = Cache(new + old, H, D, 11)
    qo = phs.kv_write_paged(r.pool, k, v, dev(c.table), dev(c.lens), cu_seqlens=dev(cu), rope=rope,
                            q=q, status=st)
    assert int(st.item()) == 0
    pos = torch.cat([torch.arange(int(o), int(o + n)) for o, n in zip(old, new)]).int().cuda()
    qr, kr = phs.rope_rotate(q, k, pos, rope)
    assert torch.equal(qo, qr)
    for got, want in ((c, k), (r, kr)):
        for b, n in enumerate(new):
            lo, hi = int(old[b]), int(old[b] + n)
            rows = slice(int(cu[b]), int(cu[b + 1]))
            assert torch.equal(got.rows(got.pool.k, b, lo, hi), want[rows])
            assert torch.equal(got.rows(got.pool.v, b, lo, hi), v[rows])
            # back to what was there: nothing else was touched
            t = np.arange(lo, hi)
            page = torch.from_numpy(got.table[b][t // 16].astype(np.int64)).cuda()
            slot = torch.from_numpy(t % 16).cuda()
            for x, y in ((got.pool.k, got.start.k), (got.pool.v, got.start.v)):
                x[page, :, slot] = y[page, :, slot]
        assert same(got.pool, got.start)


def test_write_tokens_as_append():
    lens = np.array([1, 15, 16, 17, 0, 200, 2048], np.int32)
    H, D, B = 4, 64, len(lens)
    c = Cache(np.maximum(lens, 1), H, D, 5)
    k, v, q = bf16((B, H, D), 1), bf16((B, H, D), 2), bf16((B, 8, D), 3)
    st = status()
    phs.kv_write_paged(c.pool, k, v, dev(c.table), dev(lens), status=st)
    phs.kv_append_paged(c.start, k, v, dev(c.table), dev(lens))
    assert int(st.item()) == 0 and same(c.pool, c.start)
    rope = phs.Rope.make(32, interleaved=True)
    out = torch.full((B, 8, D), 9.0, dtype=torch.bfloat16, device="cuda")
    assert phs.kv_write_paged(c.pool, k, v, dev(c.table), dev(lens), q=q, q_out=out, rope=rope,
                              status=st) is out
    qr, kr = phs.rope_rotate(q, k, dev(lens - 1), rope)
    phs.kv_append_paged(c.start, kr, v, dev(c.table), dev(lens))
    qr[4] = 0   # inactive
    assert int(st.item()) == 0 and same(c.pool, c.start) and torch.equal(out, qr)


def test_queries_rotated_in_place():
    lens = np.array([3, 40, 16], np.int32)
    H, D, T = 2, 128, 20
    cu, c = dev(np.array([0, 3, 9, 20])), Cache(lens, H, D, 6)
    k, v, q = bf16((T, H, D), 1), bf16((T, H, D), 2), bf16((T, 6, D), 3)
    a = (c.pool, k, v, dev(c.table), dev(lens))
    rope = phs.Rope.make(64)
    want = phs.kv_write_paged(*a, cu_seqlens=cu, rope=rope, q=q)
    assert phs.kv_write_paged(*a, cu_seqlens=cu, rope=rope, q=q, q_out=q) is q
    assert torch.equal(q, want)


@pytest.mark.parametrize("H,D,inter,rotary", [(8, 128, False, 128), (3, 64, True, 64),
                                              (5, 128, True, 32), (1, 64, False, 0)])
@pytest.mark.parametrize("hot", [0, 1, 40])
def test_write_8bit(H, D, inter, rotary, hot):
    """Blocks of new tokens, of earlier ones and of both, bit for bit as a bf16
    write of all tokens and the block quantiser give them."""
    old = np.array([0, 5, 31, 32, 100, 333, 64, 7], np.int32)
    new = np.array([1, 100, 1, 64, 0, 37, 31, 700], np.int32)
    lens = old + new
    before = np.maximum(old - hot, 0) // 32 * 32
    before[5] = 32                       # more earlier blocks than the rule would leave
    after = np.maximum(lens - hot, 0) // 32 * 32
    c, w = (Cache(lens, H, D, 21, qlens=np.maximum(after, 0)) for _ in range(2))
    T, B = int(new.sum()), len(new)
    cu = dev(np.concatenate([[0], np.cumsum(new)]))
    k, v, q = strided(bf16((T, H, D), 1), 8), bf16((T, H, D), 2), bf16((T, H, D), 3)
    k[3] = 0                             # a token of zeros
    k[40:72], v[40:72] = 0, 0            # blocks of zeros among them
    v[100:140, 0] *= 1e-39               # scales whose inverse overflows
    rope = phs.Rope.make(rotary, interleaved=inter) if rotary else None
    st = status()
    most = int((after - before).max()) // 32
    qo = phs.kv_write_paged(c.pool, k, v, dev(c.table), dev(lens), cu_seqlens=cu,
                            q=q if rope else None, rope=rope, int8=c.int8, qtable=dev(c.qtable),
                            qlens_before=dev(before), qlens=dev(after), max_qblocks=most, status=st)
    assert int(st.item()) == 0
    qw = phs.kv_write_paged(w.pool, k, v, dev(c.table), dev(lens), cu_seqlens=cu,
                            q=q if rope else None, rope=rope, status=st)
    phs.kv_quant_int8_block32(w.pool, dev(c.table), w.int8, dev(c.qtable), dev(before // 32),
                              dev((after - before) // 32), most, status=st)
    assert int(st.item()) == 0
    if rope:
        assert torch.equal(qo, qw)
    for a, b in ((c.int8.k, w.int8.k), (c.int8.v, w.int8.v), (c.int8.k_scale, w.int8.k_scale),
                 (c.int8.v_scale, w.int8.v_scale)):
        assert torch.equal(a, b)
    codes = c.int8.codes()
    for b in range(B):                   # and against the definition
        for j in range(int(before[b]) // 32, int(after[b]) // 32):
            for x, scale, got in ((w.pool.k, c.int8.k_scale, codes[0]),
                                  (w.pool.v, c.int8.v_scale, codes[1])):
                rows = w.rows(x, b, 32 * j, 32 * j + 32)
                for h in range(0, H, 4):
                    y, s = ref.quantise(rows[:, h])
                    p = c.qtable[b][j]
                    assert float(scale[p, h]) == float(s)
                    assert np.array_equal(got[p, h].cpu().numpy(), y)
        # tokens above the 8-bit ones are in their pages, below nothing was written there
        cold = max(int(after[b]), int(old[b]))
        for x, y, z in ((c.pool.k, w.pool.k, c.start.k), (c.pool.v, w.pool.v, c.start.v)):
            assert torch.equal(c.rows(x, b, cold, int(lens[b])), c.rows(y, b, cold, int(lens[b])))
            assert torch.equal(c.rows(x, b, 0, cold), c.rows(z, b, 0, cold))


@pytest.mark.parametrize("Hq,H,D,inter,rotary", [(32, 8, 128, False, 128), (5, 5, 128, True, 48),
                                                 (7, 1, 64, False, 64), (1, 1, 64, True, 16),
                                                 (6, 3, 128, False, 64)])
def test_queries_that_go_with_their_blocks(Hq, H, D, inter, rotary):
    """With enough blocks in the grid (max_qblocks is only a limit) the blocks'
    launch turns the queries of their new tokens: nothing that comes out differs,
    of a request that is refused and of one with a block outside the pool neither."""
    old = np.array([0, 5, 31, 32, 100, 333, 64, 7], np.int32)
    new = np.array([1, 100, 1, 64, 0, 37, 31, 700], np.int32)
    lens, hot = old + new, np.array([0, 1, 40, 0, 0, 0, 70, 13])
    before, after = (np.maximum(n - hot, 0) // 32 * 32 for n in (old, lens))
    T, cu = int(new.sum()), np.concatenate([[0], np.cumsum(new)])
    k, v = strided(bf16((T, H, D), 1), 8), bf16((T, H, D), 2)
    q = strided(bf16((T, Hq, D), 3), 16)
    rope = phs.Rope.make(rotary, interleaved=inter)
    pos = torch.cat([torch.arange(int(o), int(o + n)) for o, n in zip(old, new)]).int().cuda()
    want = phs.rope_rotate(q, None, pos, rope)[0]

    def call(most, lens, qtable_of):
        c, st = Cache(old + new, H, D, 21, qlens=np.maximum(after, 32)), status()
        for x in (c.int8.k, c.int8.v, c.int8.k_scale, c.int8.v_scale):
            x.zero_()
        out = torch.full((T + 2, Hq, D), 9.0, dtype=torch.bfloat16, device="cuda")
        got = phs.kv_write_paged(c.pool, k, v, dev(c.table), dev(lens), cu_seqlens=dev(cu), q=q,
                                 q_out=out[:T], rope=rope, int8=c.int8,
                                 qtable=dev(qtable_of(c.qtable)), qlens_before=dev(before),
                                 qlens=dev(after), max_qblocks=most, status=st)
        assert bool((out[T:] == 9).all())
        return c, got, int(st.item())

    def check(lens, qtable_of, want, code):
        few, many = (call(most, lens, qtable_of) for most in (int((after - before).max()) // 32, 200))
        for c, got, st in (few, many):
            assert st == code and torch.equal(got, want)
        a, b = few[0], many[0]
        assert same(a.pool, b.pool)
        for x, y in ((a.int8.k, b.int8.k), (a.int8.v, b.int8.v), (a.int8.k_scale, b.int8.k_scale),
                     (a.int8.v_scale, b.int8.v_scale)):
            assert torch.equal(x, y)

    check(lens, lambda t: t, want, 0)

    def missing(t):
        t = t.copy()
        t[7, 3] = -1
        return t

    check(lens, missing, want, -3)
    refused = lens.copy()
    refused[7] = 699                     # below its new tokens
    zero = want.clone()
    zero[int(cu[7]):] = 0
    check(refused, lambda t: t, zero, -3)


def test_write_8bit_tokens():
    """One token at a time: a block is quantised when its last token is old
    enough, wholly from pages, or with the new token as its last."""
    H, D, B = 2, 64, 3
    final = np.array([70, 97, 40], np.int32)
    hots = np.array([0, 5, 33])
    end = np.maximum(final - hots, 0) // 32 * 32
    c, w = (Cache(final, H, D, 31, qlens=np.maximum(end, 32)) for _ in range(2))
    rope = phs.Rope.make(64)
    st = status()
    for step in range(70, 0, -1):
        lens = final - step + 1
        was, now = (np.where(n > 0, np.maximum(n - hots, 0) // 32 * 32, 0) for n in (lens - 1, lens))
        lens = np.maximum(lens, 0)
        k, v = bf16((B, H, D), 100 + step), bf16((B, H, D), 200 + step)
        phs.kv_write_paged(c.pool, k, v, dev(c.table), dev(lens), rope=rope, int8=c.int8,
                           qtable=dev(c.qtable), qlens_before=dev(was), qlens=dev(now),
                           max_qblocks=1, status=st)
        phs.kv_write_paged(w.pool, k, v, dev(c.table), dev(lens), rope=rope, status=st)
    phs.kv_quant_int8_block32(w.pool, dev(c.table), w.int8, dev(c.qtable), dev(np.zeros(B)),
                              dev(end // 32), 2, status=st)
    assert int(st.item()) == 0
    for b in range(B):
        p = torch.from_numpy(c.qtable[b][:end[b] // 32].astype(np.int64)).cuda()
        assert torch.equal(c.int8.k[p], w.int8.k[p]) and torch.equal(c.int8.v[p], w.int8.v[p])
        assert torch.equal(c.rows(c.pool.k, b, int(end[b]), int(final[b])),
                           w.rows(w.pool.k, b, int(end[b]), int(final[b])))


@pytest.mark.parametrize("H,D", [(8, 128), (3, 64), (1, 128)])
def test_read_back(H, D):
    lens = np.array([300, 33, 64, 5, 100], np.int32)
    qlens = np.array([256, 32, 64, 0, 32], np.int32)
    starts = np.array([3, 20, 63, 5, 31], np.int32)
    count = np.array([290, 13, 1, 0, 40], np.int32)
    c = Cache(lens, H, D, 41, qlens=qlens)
    cu = np.concatenate([[2], 2 + np.cumsum(count)])      # rows of no request around them
    T = int(cu[-1]) + 3
    st = status()
    ko, vo = (torch.full((T, H, D), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    got = phs.kv_read_paged(c.pool, dev(c.table), dev(starts), dev(cu), T, 290, int8=c.int8,
                            qtable=dev(c.qtable), qlens=dev(qlens), k_out=ko, v_out=vo, status=st)
    assert got[0] is ko and got[1] is vo and int(st.item()) == 0
    codes = c.int8.codes()
    for x, scale, code, out in ((c.pool.k, c.int8.k_scale, codes[0], ko),
                                (c.pool.v, c.int8.v_scale, codes[1], vo)):
        assert bool((out[:2] == 5).all()) and bool((out[int(cu[-1]):] == 5).all())
        for b in range(len(lens)):
            for i in range(int(count[b])):
                t = int(starts[b]) + i
                if t < qlens[b]:
                    p = c.qtable[b][t // 32]
                    want = (code[p, :, t % 32].float() * scale[p][:, None]).bfloat16()
                else:
                    want = x[c.table[b][t // 16], :, t % 16]
                assert torch.equal(out[int(cu[b]) + i], want), (b, t)
    # without the 8-bit blocks all tokens come from their pages
    k2, v2 = phs.kv_read_paged(c.pool, dev(c.table), dev(starts), dev(cu), T, 290, status=st)
    assert torch.equal(k2[2:292], c.rows(c.pool.k, 0, 3, 293))
    assert torch.equal(v2[2:292], c.rows(c.pool.v, 0, 3, 293)) and int(st.item()) == 0


def test_written_cache_is_what_decode_attends_to():
    """A prompt written in two parts, half of it in 8 bits, then a decode step
    over it: as over a cache of single appends and the block quantiser."""
    H, D, Hq, n = 2, 128, 8, 500
    c, w = (Cache([n + 1], H, D, 51, qlens=[320]) for _ in range(2))
    k, v, q = bf16((n + 1, H, D), 1), bf16((n + 1, H, D), 2), bf16((n + 1, Hq, D), 3)
    rope = phs.Rope.make(128)
    qr, kr = phs.rope_rotate(q, k, torch.arange(n + 1, dtype=torch.int32, device="cuda"), rope)
    st = status()
    at = 0
    for upto, b0, b1 in ((200, 0, 160), (n, 160, 320)):
        phs.kv_write_paged(c.pool, k[at:upto], v[at:upto], dev(c.table), dev([upto]),
                           cu_seqlens=dev([0, upto - at]), rope=rope, int8=c.int8,
                           qtable=dev(c.qtable), qlens_before=dev([b0]), qlens=dev([b1]),
                           max_qblocks=5, status=st)
        at = upto
    for t in range(n):
        phs.kv_append_paged(w.pool, kr[t:t + 1], v[t:t + 1], dev(w.table), dev([t + 1]), status=st)
    phs.kv_quant_int8_block32(w.pool, dev(w.table), w.int8, dev(w.qtable), dev([0]), dev([10]), 10,
                              status=st)
    outs = [phs.attn_decode_full_paged(qr[n:], x.pool, dev(x.table), dev([n + 1]), n + 1,
                                       int8=x.int8, qtable=dev(x.qtable), qlens=dev([320]),
                                       k_new=kr[n:], v_new=v[n:], status=st) for x in (c, w)]
    assert int(st.item()) == 0 and torch.equal(*outs)


# ------------------------------------------------------------ bad device data --
def write_case():
    H, D = 2, 64
    c = Cache([40, 20, 70], H, D, 61, qlens=[32, 0, 64])
    cu, T = [0, 10, 20, 40], 40
    k, v, q = bf16((T, H, D), 1), bf16((T, H, D), 2), bf16((T, H, D), 3)
    a = dict(cu=cu, lens=[40, 20, 70], before=[0, 0, 32], after=[32, 0, 64], table=c.table,
             qtable=c.qtable, count=None, most=1)
    return c, k, v, q, a


def run_write(c, k, v, q, a):
    st = status()
    out = torch.full_like(q, 3.0)
    phs.kv_write_paged(c.pool, k, v, dev(a["table"]), dev(a["lens"]), cu_seqlens=dev(a["cu"]), q=q,
                       q_out=out, rope=phs.Rope.make(64), int8=c.int8, qtable=dev(a["qtable"]),
                       qlens_before=dev(a["before"]), qlens=dev(a["after"]), max_qblocks=a["most"],
                       page_refcount=None if a["count"] is None else dev(a["count"]), status=st)
    return int(st.item()), out


@pytest.mark.parametrize("cu", [[0, 10, 5, 40], [-1, 10, 20, 40], [0, 10, 20, 41], [0, 50, 20, 40]])
def test_bad_ranges_refuse_the_write(cu):
    c, k, v, q, a = write_case()
    code, out = run_write(c, k, v, q, a | dict(cu=cu))
    assert code == -3 and bool((out == 3).all()) and same(c.pool, c.start)
    assert torch.equal(c.int8.k, c.int8_start.k) and torch.equal(c.int8.v_scale, c.int8_start.v_scale)


@pytest.mark.parametrize("bad", [
    dict(lens=[9, 20, 70], before=[0, 0, 32], after=[0, 0, 64]), dict(before=[-32, 0, 32]),
    dict(after=[31, 0, 64]), dict(after=[64, 0, 64]), dict(before=[32, 0, 32]),
    dict(before=[32, 0, 32], after=[0, 0, 64]), dict(lens=[100, 20, 70], after=[96, 0, 64])])
def test_bad_lengths_refuse_the_request(bad):
    """Request 0 is left out, the others come out as always."""
    c, k, v, q, a = write_case()
    code, out = run_write(c, k, v, q, a | bad)
    w, *_ = write_case()
    ok, want = run_write(w, k, v, q, a)
    assert code == -3 and ok == 0
    assert not out[:10].any() and torch.equal(out[10:], want[10:])
    for b, lo, hi in ((0, 0, 40),):
        assert torch.equal(c.rows(c.pool.k, b, lo, hi), c.rows(c.start.k, b, lo, hi))
    p0, p2 = c.qtable[0][0], c.qtable[2][1]
    assert torch.equal(c.int8.k[p0], c.int8_start.k[p0])
    assert torch.equal(c.int8.k[p2], w.int8.k[p2]) and torch.equal(c.int8.v[p2], w.int8.v[p2])
    assert torch.equal(c.rows(c.pool.v, 1, 10, 20), w.rows(w.pool.v, 1, 10, 20))


def test_bad_pages_are_not_written():
    c, k, v, q, a = write_case()
    table, qtable = c.table.copy(), c.qtable.copy()
    table[1][1], table[0][2], qtable[2][1] = 10**6, -1, 10**6
    code, out = run_write(c, k, v, q, a | dict(table=table, qtable=qtable))
    w, *_ = write_case()
    _, want = run_write(w, k, v, q, a)
    assert code == -3 and torch.equal(out, want)
    assert torch.equal(c.rows(c.pool.k, 1, 10, 16), w.rows(w.pool.k, 1, 10, 16))
    assert torch.equal(c.rows(c.pool.k, 1, 16, 20), c.rows(c.start.k, 1, 16, 20))
    assert torch.equal(c.rows(c.pool.k, 0, 32, 40), c.rows(c.start.k, 0, 32, 40))
    p0, p2 = c.qtable[0][0], c.qtable[2][1]
    assert torch.equal(c.int8.k[p0], w.int8.k[p0])
    assert torch.equal(c.int8.k[p2], c.int8_start.k[p2])
    # an earlier token's page that is missing: its block is left out
    c, k, v, q, a = write_case()
    table = c.table.copy()
    table[0][0] = -1
    code, _ = run_write(c, k, v, q, a | dict(table=table))
    assert code == -3 and torch.equal(c.int8.k[p0], c.int8_start.k[p0])
    assert torch.equal(c.int8.k[p2], w.int8.k[p2])
    # a table that ends before the tokens
    c, k, v, q, a = write_case()
    code, _ = run_write(c, k, v, q, a | dict(table=c.table[:, :2].copy()))
    assert code == -3
    assert torch.equal(c.rows(c.pool.k, 1, 10, 20), w.rows(w.pool.k, 1, 10, 20))


def test_shared_pages_are_not_written():
    c, k, v, q, a = write_case()
    count = np.ones(c.pool.k.shape[0], np.int32)
    count[c.table[1][0]] = 2
    code, out = run_write(c, k, v, q, a | dict(count=count))
    w, *_ = write_case()
    _, want = run_write(w, k, v, q, a)
    assert code == -4 and torch.equal(out, want)
    assert torch.equal(c.rows(c.pool.k, 1, 10, 16), c.rows(c.start.k, 1, 10, 16))
    assert torch.equal(c.rows(c.pool.k, 1, 16, 20), w.rows(w.pool.k, 1, 16, 20))


def test_bad_reads():
    H, D = 2, 64
    c = Cache([40, 70], H, D, 71, qlens=[32, 32])

    def read(cu=(0, 20, 50), starts=(10, 40), qlens=(32, 32), table=c.table, most=30):
        st = status()
        k, v = (torch.full((50, H, D), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        phs.kv_read_paged(c.pool, dev(table), dev(starts), dev(cu), 50, most, int8=c.int8,
                          qtable=dev(c.qtable), qlens=dev(qlens), k_out=k, v_out=v, status=st)
        return int(st.item()), k, v

    good, k, v = read()
    assert good == 0
    for cu in ((0, 30, 20), (-1, 20, 50), (0, 20, 51)):
        code, x, y = read(cu=cu)
        assert code == -3 and bool((x == 5).all()) and bool((y == 5).all())
    for kw in (dict(starts=(-1, 40)), dict(qlens=(-32, 32)), dict(qlens=(31, 32)),
               dict(starts=(2**31 - 1, 40))):
        code, x, y = read(**kw)
        assert code == -3 and bool((x[:20] == 5).all()) and torch.equal(x[20:], k[20:])
    code, x, y = read(most=25)
    assert code == -3 and torch.equal(x[:20], k[:20]) and bool((x[20:] == 5).all())
    table = c.table.copy()
    table[1][3] = 10**6                       # tokens 48..63 of request 1
    code, x, y = read(table=table)
    assert code == -3 and not x[28:44].any() and not y[28:44].any()
    x[28:44], y[28:44] = k[28:44], v[28:44]
    assert torch.equal(x, k) and torch.equal(y, v)


def test_refusals_of_the_binding():
    H, D = 2, 64
    c = Cache([4], H, D, 81, qlens=[0])
    k, i = bf16((4, H, D), 1), dev([4])
    t, cu = dev(c.table), dev([0, 4])
    ok = dict(cu_seqlens=cu)
    rope = phs.Rope.make(64)
    for bad in (dict(k=k.float()), dict(k=k[:, :1]), dict(k=k.transpose(0, 1)), dict(k=k[..., ::2]),
                dict(v=k[:3]), dict(table=t.long()), dict(lens=dev([4, 4])),
                dict(cu_seqlens=dev([0, 4, 4])), dict(cu_seqlens=None), dict(q=k), dict(q_out=k),
                dict(q=k[:2], rope=rope), dict(q=k, rope=rope, q_out=k[:2]),
                dict(rope=phs.Rope(rope.turns.int())), dict(qlens=i), dict(int8=c.int8),
                dict(int8=c.int8, qtable=t, qlens=i, qlens_before=dev([0, 0])),
                dict(page_refcount=dev([1])), dict(k=k.cpu())):
        a = dict(k=k, v=k, table=t, lens=i) | ok | bad
        with pytest.raises((ValueError, TypeError)):
            phs.kv_write_paged(c.pool, a.pop("k"), a.pop("v"), a.pop("table"), a.pop("lens"), **a)
    with pytest.raises(phs.PhsError):      # rows that do not begin on 16 bytes
        phs.kv_write_paged(c.pool, strided(k, 4), k, t, i, cu_seqlens=cu)
    with pytest.raises(phs.PhsError):      # a part that is no multiple of 16
        phs.rope_rotate(k, None, dev([0, 1, 2, 3]), phs.Rope.make(8))
    assert same(c.pool, c.start)
