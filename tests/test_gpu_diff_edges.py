"""Differential attention decode with values that are not finite, or hardly
above zero."""
import pytest
import torch

import paged_hybrid_sliding_gb300 as phs
from gpu_util import dev
from test_gpu_diff import check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,H,Hv", [(64, 4, 2), (128, 4, 2), (64, 12, 1)])
@pytest.mark.parametrize("tps", [32, 128, 4096])   # many splits, a few, one
@pytest.mark.parametrize("norm", [True, False])
def test_a_nan_query_gives_nan_however_the_request_is_split(D, H, Hv, tps, norm):
    """NaN in the query of either map or of both: the head's row is NaN, in every
    column, and the other heads and requests are as without it."""
    lens = [700, 300, 90]
    pool, q, bt, lens, w = make(lens, H, Hv, D, 21, norm=norm)
    args = (pool, dev(bt), dev(lens), 700, w)
    kw = dict(out_dtype=torch.float32, tokens_per_split=tps)
    want = phs.attn_decode_diff_paged(q, *args, **kw)
    bad = q.clone()
    bad[0, 0, 5] = float("nan")              # request 0, head 0: first map
    bad[1, 2 * (H - 1) + 1] = float("nan")   # request 1, last head: second map
    bad[2, 2:4] = float("nan")               # request 2, head 1: both
    out = phs.attn_decode_diff_paged(bad, *args, **kw)
    for b, i in ((0, 0), (1, H - 1), (2, 1)):
        assert torch.isnan(out[b, i]).all(), (b, i)
        want[b, i] = out[b, i] = 0
    assert torch.equal(out, want)


@pytest.mark.parametrize("tps", [32, 4096])
def test_a_nan_key_gives_nan_however_the_request_is_split(tps):
    pool, q, bt, lens, w = make([700, 300], 4, 2, 64, 22)
    kw = dict(out_dtype=torch.float32, tokens_per_split=tps)
    want = phs.attn_decode_diff_paged(q, pool, dev(bt), dev(lens), 700, w, **kw)
    pool.k[int(bt[0, 20]), 3, 4, 7] = float("nan")   # value head 1, second map
    out = phs.attn_decode_diff_paged(q, pool, dev(bt), dev(lens), 700, w, **kw)
    assert torch.isnan(out[0, 2:]).all()
    assert torch.equal(out[0, :2], want[0, :2]) and torch.equal(out[1], want[1])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [9, 500])
def test_norm_of_rows_whose_squares_underflow(D, n):
    """Values of 2^-85: their squares are zero in fp32, they themselves are not,
    and the root of eps is what the norm divides by."""
    pool, q, bt, lens, w = make([n], 4, 2, D, 23)
    pool.v.mul_(2.0**-85)
    out = phs.attn_decode_diff_paged(q, pool, dev(bt), dev(lens), n, w, out_dtype=torch.float32)
    check(out, pool, q, bt, lens, w)
    assert bool((out != 0).any())
    # with eps 0 and no value at all the row is zero
    pool.v.zero_()
    w.norm_eps = 0.0
    out = phs.attn_decode_diff_paged(q, pool, dev(bt), dev(lens), n, w, out_dtype=torch.float32)
    assert not out.any()
