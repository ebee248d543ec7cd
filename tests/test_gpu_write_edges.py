"""Cache writes with values that are not finite, and calls that hold one long
prompt beside many single tokens."""
import numpy as np
import pytest
import torch

import paged_hybrid_sliding_gb300 as phs
from gpu_util import dev
from test_gpu_write import Cache, bf16, same, status

pytestmark = pytest.mark.gpu


def int8_tensors(pool):
    return pool.k, pool.v, pool.k_scale, pool.v_scale


def same_bits(a, b):
    if a.dtype.is_floating_point:
        a, b = (t.view(torch.int32 if t.dtype == torch.float32 else torch.int16) for t in (a, b))
    return torch.equal(a, b)


@pytest.mark.parametrize("D,rotary", [(64, 64), (128, 32)])
def test_8bit_blocks_of_values_that_are_not_finite(D, rotary):
    """Infinities and NaN give the bytes that a bf16 write and the block
    quantiser give, and stay in their block and head."""
    H, lens = 3, np.array([160, 70], np.int32)
    after, T = np.array([160, 64], np.int32), 230
    cu, rope = dev(np.array([0, 160, 230])), phs.Rope.make(rotary)
    k, v, q = bf16((T, H, D), 1), bf16((T, H, D), 2), bf16((T, 2 * H, D), 3)
    clean = [t.clone() for t in (k, v, q)]
    k[40, 1, 3], k[41, 1, D - 1], k[70, 0, 5] = float("inf"), float("nan"), float("-inf")
    v[100, 2, 7], v[101, 2, 8], v[170, 0, 9] = float("nan"), float("-inf"), float("inf")
    v[130:160, 1] = float("nan")
    q[5, 4, 2] = float("nan")
    runs = []
    for kk, vv, qq in ((k, v, q), clean):
        for blocks in (5, 400):      # (with more the blocks' launch turns the queries)
            c, st = Cache(lens, H, D, 21, qlens=after), status()
            out = phs.kv_write_paged(c.pool, kk, vv, dev(c.table), dev(lens), cu_seqlens=cu, rope=rope,
                                     q=qq, int8=c.int8, qtable=dev(c.qtable), qlens_before=dev([0, 0]),
                                     qlens=dev(after), max_qblocks=blocks, status=st)
            assert int(st.item()) == 0
            runs.append((c, out))
    w, st = Cache(lens, H, D, 21, qlens=after), status()
    want = phs.kv_write_paged(w.pool, k, v, dev(w.table), dev(lens), cu_seqlens=cu, rope=rope, q=q,
                              status=st)
    phs.kv_quant_int8_block32(w.pool, dev(w.table), w.int8, dev(w.qtable), dev([0, 0]),
                              dev(after // 32), 5, status=st)
    assert int(st.item()) == 0
    for c, out in runs[:2]:
        assert same_bits(out, want)
        for a, b in zip(int8_tensors(c.int8), int8_tensors(w.int8)):
            assert same_bits(a, b)
    # other blocks and heads hold what they hold without these values
    bad, good = runs[0][0], runs[2][0]
    hit = {(0, 1, 1), (0, 2, 0), (0, 3, 2), (0, 4, 1), (1, 0, 0)}     # request, block, head
    for b in range(2):
        for j in range(int(after[b]) // 32):
            for h in range(H):
                if (b, j, h) not in hit:
                    p = bad.qtable[b][j]
                    for x, y in zip(int8_tensors(bad.int8), int8_tensors(good.int8)):
                        assert torch.equal(x[p, h], y[p, h]), (b, j, h)


@pytest.mark.parametrize("H,D,Hq", [(2, 64, 4), (4, 128, 16)])
def test_a_long_prompt_beside_many_tokens(H, D, Hq):
    """One call gives what the prompt's and the tokens' own calls give, written
    and read back."""
    rng = np.random.default_rng(D)
    n_long, B = 3001, 70
    new = np.ones(B, np.int32)
    new[33] = n_long
    old = rng.integers(0, 300, B).astype(np.int32)
    old[33] = 45
    lens = old + new
    before, after = (np.maximum(n - 20, 0) // 32 * 32 for n in (old, lens))
    # (some tokens complete a block)
    T, cu = int(new.sum()), np.concatenate([[0], np.cumsum(new)])
    k, v, q = bf16((T, H, D), 1), bf16((T, H, D), 2), bf16((T, Hq, D), 3)
    rope, most = phs.Rope.make(D), int((after - before).max()) // 32
    assert ((after - before)[np.arange(B) != 33] > 0).any()
    c, w = (Cache(lens, H, D, 5, qlens=np.maximum(after, 32)) for _ in range(2))
    st = status()

    def write(cache, rows, reqs, most):
        sub = np.concatenate([[0], np.cumsum(new[reqs])])
        return phs.kv_write_paged(
            cache.pool, k[rows], v[rows], dev(cache.table[reqs]), dev(lens[reqs]), cu_seqlens=dev(sub),
            rope=rope, q=q[rows], int8=cache.int8, qtable=dev(cache.qtable[reqs]),
            qlens_before=dev(before[reqs]), qlens=dev(after[reqs]), max_qblocks=most, status=st)

    def read(cache, reqs):
        sub = np.concatenate([[0], np.cumsum(new[reqs])])
        return phs.kv_read_paged(cache.pool, dev(cache.table[reqs]), dev(old[reqs]), dev(sub),
                                 int(sub[-1]), int(new[reqs].max()), int8=cache.int8,
                                 qtable=dev(cache.qtable[reqs]), qlens=dev(after[reqs]), status=st)

    everything = np.arange(B)
    got, back = write(c, slice(None), everything, most), read(c, everything)
    for lo, hi in ((0, 33), (33, 34), (34, B)):
        reqs, rows = everything[lo:hi], slice(int(cu[lo]), int(cu[hi]))
        m = int((after - before)[reqs].max()) // 32
        assert torch.equal(write(w, rows, reqs, m), got[rows])
        for x, y in zip(read(w, reqs), back):
            assert torch.equal(x, y[rows])
    assert int(st.item()) == 0 and same(c.pool, w.pool)
    for a, b in zip(int8_tensors(c.int8), int8_tensors(w.int8)):
        assert torch.equal(a, b)


def test_reads_near_the_last_position():
    """A start near 2^31 beside a longer request: its pages are outside the
    table, its rows zero, the other's rows what they are."""
    H, D = 2, 64
    c, st = Cache(np.array([400, 400], np.int32), H, D, 3), status()
    for start, n in ((2**31 - 100, 60), (2**31 - 17 - 33, 33), (2**31 - 18, 1)):
        k, v = phs.kv_read_paged(c.pool, dev(c.table), torch.tensor([5, start], dtype=torch.int32).cuda(),
                                 dev([0, 390, 390 + n]), 390 + n, 390, status=st)
        assert int(st.item()) == -3 and not k[390:].any() and not v[390:].any()
        assert torch.equal(k[:390], c.rows(c.pool.k, 0, 5, 395))
        assert torch.equal(v[:390], c.rows(c.pool.v, 0, 5, 395))
    st.zero_()   # one further on the range itself is refused
    k = torch.full((391, H, D), 3.0, dtype=torch.bfloat16, device="cuda")
    phs.kv_read_paged(c.pool, dev(c.table), torch.tensor([5, 2**31 - 17], dtype=torch.int32).cuda(),
                      dev([0, 390, 391]), 391, 390, k_out=k, v_out=k.clone(), status=st)
    assert int(st.item()) == -3 and bool((k[390:] == 3).all())
