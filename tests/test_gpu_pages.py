"""Device-side page operations against plain loops: every table entry, count
and page byte equal."""
import numpy as np
import pytest
import torch

import ops_ref
import paged_hybrid_sliding_gb300 as phs
import synth
from gpu_util import dev

pytestmark = pytest.mark.gpu


class Cache:
    """A pool, block table, lengths and counts on host and device."""

    def __init__(self, lens, num_pages, seed, layers=2, heads=2, dim=64, width=None, shared=0):
        rs = np.random.RandomState(seed)
        self.lens = np.asarray(lens, np.int32)
        need = [ops_ref.pages(n) for n in self.lens]
        width = width or max(need + [1]) + 1
        ids = rs.permutation(num_pages)
        self.table = np.full((len(lens), width), -7, np.int32)
        self.counts = np.zeros(num_pages, np.int32)
        at = shared
        for r, k in enumerate(need):
            c = min(shared, k)
            self.table[r, :c] = ids[:c]
            self.table[r, c:k] = ids[at:at + k - c]
            at += k - c
            self.counts[self.table[r, :k]] += 1
        self.pools = [phs.PagedPool(
            synth.normal_bf16((num_pages, heads, 16, dim), seed + 10 * l, device="cuda"),
            synth.normal_bf16((num_pages, heads, 16, dim), seed + 10 * l + 1, device="cuda"))
            for l in range(layers)]
        self.host = [(synth.bits(p.k).copy(), synth.bits(p.v).copy()) for p in self.pools]
        self.d_table, self.d_lens, self.d_counts = dev(self.table), dev(self.lens), dev(self.counts)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def free(self, rows, host=True):
        phs.pages_free(self.d_table, self.d_lens, self.d_counts, dev(rows), status=self.status)
        if host:
            ops_ref.free_rows(self.table, self.lens, self.counts, rows)

    def fork(self, src, dst, host=True):
        phs.pages_fork(self.pools, self.d_table, self.d_lens, self.d_counts, dev(src), dev(dst),
                       status=self.status)
        if host:
            ops_ref.fork_rows(self.host, self.table, self.lens, self.counts, src, dst)

    def check(self, code=0, data_below=None):
        torch.cuda.synchronize()
        assert int(self.status.item()) == code
        self.status.zero_()
        np.testing.assert_array_equal(self.d_lens.cpu().numpy(), self.lens)
        np.testing.assert_array_equal(self.d_counts.cpu().numpy(), self.counts)
        np.testing.assert_array_equal(self.d_table.cpu().numpy(), self.table)
        for p, (k, v) in zip(self.pools, self.host):
            np.testing.assert_array_equal(synth.bits(p.k), k)
            np.testing.assert_array_equal(synth.bits(p.v), v)


@pytest.mark.parametrize("heads,dim,layers", [(1, 64, 1), (2, 128, 3), (5, 64, 2), (1, 64, 65)])
def test_fork_and_free(heads, dim, layers):
    # lengths 1, 15, 16, 17, 0 (an empty request), a long one; three free rows
    c = Cache([1, 15, 16, 17, 0, 333, 0, 0, 0, 0], 64, 3, layers=layers, heads=heads, dim=dim)
    c.fork([5, 0, 2, 4], [7, 6, 9, 8])
    c.check()
    c.free([5, 7, 4])
    c.check()
    c.fork([1, 3, 6], [5, 7, 4])
    c.check()
    c.free([0, 1, 2, 3, 4, 5, 6, 7, 8, 9])
    c.check()
    assert not c.counts.any()


def test_fork_many_children_of_one_row_and_of_each_other():
    n = 300   # a full block of the plan plus a tail
    c = Cache([100] + [0] * n, 800, 5, layers=1)
    c.fork([0] * 150, list(range(1, 151)))
    c.check()
    c.fork(list(range(1, 151)), list(range(n, 150, -1)))
    c.check()


def test_fork_over_many_entries_and_scattered_free_pages():
    rows = 1500
    lens = [(7 * r) % 40 + 1 for r in range(rows)] + [0] * rows
    c = Cache(lens, 9000, 7, layers=1, heads=1)
    rs = np.random.RandomState(1)
    c.fork(list(rs.permutation(rows)), [rows + r for r in rs.permutation(rows)])
    c.check()


def test_fork_refusals_leave_the_others_done():
    c = Cache([20, 40, 0, 0, 0, 5], 16, 9)
    # 0 -> 2 is good; 1 -> 5 not free; 1 -> 2 listed before; 9 out of range;
    # 2 is a source and a destination; 1 -> 4 is good
    before = c.table.copy()
    c.fork([0, 1, 1, 9], [2, 5, 2, 3], host=False)
    ops_ref.fork_rows(c.host, c.table, c.lens, c.counts, [0], [2])
    torch.cuda.synchronize()
    assert int(c.status.item()) in (-1, -3)
    c.status.zero_()
    c.check()
    c.fork([3, 1], [4, 3], host=False)   # row 3 is a source: refused
    ops_ref.fork_rows(c.host, c.table, c.lens, c.counts, [3], [4])
    c.check(-1)
    assert (c.table[5] == before[5]).all()


def test_fork_without_a_page_left():
    c = Cache([17, 33, 16, 0, 0, 0, 0], 8, 11)   # 2 + 3 + 1 pages: 2 free
    c.fork([0, 1, 0, 2], [3, 4, 5, 6], host=False)
    # the third entry needs a page and there is none; the fourth needs none
    ops_ref.fork_rows(c.host, c.table, c.lens, c.counts, [0, 1, 2], [3, 4, 6])
    c.check(-11)


def test_free_refusals():
    c = Cache([20, 40, 5], 16, 13)
    c.free([1, 1, 7, -1], host=False)
    ops_ref.free_rows(c.table, c.lens, c.counts, [1])
    torch.cuda.synchronize()
    assert int(c.status.item()) in (-1, -3)
    c.status.zero_()
    c.check()
    # a table entry outside the pool, and one whose page is not live
    dead = int(np.flatnonzero(c.counts == 0)[0])
    c.table[0, 0], c.table[2, 0] = 99, dead
    c.d_table.copy_(dev(c.table))
    c.free([0, 2], host=False)
    c.counts[c.table[0, 1]] -= 1
    c.lens[0] = c.lens[2] = 0
    c.check(-3)


def test_a_length_outside_the_table_is_recorded():
    c = Cache([20, 40, 0, 0], 16, 15)
    c.d_lens.copy_(dev([-3, 999, 0, 0]))
    c.lens[:] = [-3, 999, 0, 0]
    c.fork([0, 1], [2, 3], host=False)
    c.check(-3)
    c.free([0, 1], host=False)
    c.lens[:2] = 0
    c.check(-3)


@pytest.mark.parametrize("num_pages,lens,shared", [
    (1, [1], 0), (40, [0, 0], 0), (64, [100, 17, 16, 1, 0], 0), (64, [100, 90, 300], 4),
    (1023, [1, 900, 4000], 1), (1024, [3000, 0, 2000], 0), (5000, [16 * 2000, 16 * 999, 5], 2),
    (70, [70 * 16], 0)])
@pytest.mark.parametrize("in_place", [True, False])
def test_compact(num_pages, lens, shared, in_place):
    c = Cache(lens, num_pages, 17, shared=shared)
    old = c.table.copy(), c.counts.copy()
    outs = {} if in_place else dict(block_table_out=torch.empty_like(c.d_table),
                                    page_refcount_out=torch.empty_like(c.d_counts))
    page_map, live = phs.pages_compact(c.pools, c.d_table, c.d_lens, c.d_counts, status=c.status,
                                       **outs)
    ref_map, ref_live = ops_ref.compact(c.host, c.table, c.lens, c.counts)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(page_map.cpu().numpy(), ref_map)
    assert int(live.item()) == ref_live
    if not in_place:
        np.testing.assert_array_equal(c.d_table.cpu().numpy(), old[0])
        np.testing.assert_array_equal(c.d_counts.cpu().numpy(), old[1])
        c.d_table, c.d_counts = outs["block_table_out"], outs["page_refcount_out"]
    c.check()
    # a compact pool stays as it is
    page_map, _ = phs.pages_compact(c.pools, c.d_table, c.d_lens, c.d_counts, status=c.status)
    ids = np.arange(num_pages)
    np.testing.assert_array_equal(page_map.cpu().numpy(), np.where(ids < ref_live, ids, -1))
    c.check()


def test_compact_leaves_bad_entries():
    c = Cache([100, 40], 64, 19)
    dead = int(np.flatnonzero(c.counts == 0)[-1])
    c.table[0, 0], c.table[1, 1] = 400, dead
    c.d_table.copy_(dev(c.table))
    phs.pages_compact(c.pools, c.d_table, c.d_lens, c.d_counts, status=c.status)
    page_map, _ = ops_ref.compact(c.host, np.zeros((0, 1), np.int32), [], c.counts)
    for r in range(2):
        for j in range(ops_ref.pages(c.lens[r])):
            p = c.table[r, j]
            if 0 <= p < 64 and page_map[p] >= 0:
                c.table[r, j] = page_map[p]
    c.check(-3)


def test_captured_and_replayed_beam_steps():
    """Free, fork and compact recorded once and replayed: each replay is the
    next step on the tables as they then are."""
    c = Cache([100, 37, 64, 20], 96, 21)
    src, dst = [0, 0], [2, 3]
    ws = [torch.empty(1 << 16, dtype=torch.uint8, device="cuda") for _ in range(2)]
    d_src, d_dst = dev(src), dev(dst)

    def step():
        phs.pages_free(c.d_table, c.d_lens, c.d_counts, d_dst, status=c.status)
        phs.pages_fork(c.pools, c.d_table, c.d_lens, c.d_counts, d_src, d_dst, workspace=ws[0],
                       status=c.status)
        phs.pages_compact(c.pools, c.d_table, c.d_lens, c.d_counts, page_map=pm, num_live=nl,
                          workspace=ws[1], status=c.status)

    pm = torch.empty_like(c.d_counts)
    nl = torch.empty(1, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        g.replay()
        ops_ref.free_rows(c.table, c.lens, c.counts, dst)
        ops_ref.fork_rows(c.host, c.table, c.lens, c.counts, src, dst)
        ops_ref.compact(c.host, c.table, c.lens, c.counts)
        c.check()


def test_host_refusals():
    c = Cache([20, 0], 16, 23)
    one = dev([0])
    cases = [
        (ValueError, lambda: phs.pages_free(c.d_table, c.d_lens[:1], c.d_counts, one)),
        (ValueError, lambda: phs.pages_free(c.d_table, c.d_lens, c.d_counts, one.long())),
        (ValueError, lambda: phs.pages_free(c.d_table[:, ::2], c.d_lens, c.d_counts, one)),
        (ValueError, lambda: phs.pages_fork([], c.d_table, c.d_lens, c.d_counts, one, dev([1]))),
        (ValueError, lambda: phs.pages_fork(c.pools, c.d_table, c.d_lens, c.d_counts[:9], one,
                                            dev([1]))),
        (ValueError, lambda: phs.pages_fork(c.pools, c.d_table, c.d_lens, c.d_counts, one,
                                            dev([1, 1]))),
        (ValueError, lambda: phs.pages_compact(c.pools, c.d_table, c.d_lens, c.d_counts,
                                               block_table_out=c.d_table[:1])),
    ]
    for kind, call in cases:
        with pytest.raises(kind):
            call()
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    big = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    with pytest.raises(phs.PhsError) as e:
        phs.pages_fork(c.pools, c.d_table, c.d_lens, c.d_counts, one, dev([1]), workspace=small)
    assert e.value.code == -5
    with pytest.raises(phs.PhsError) as e:
        phs.pages_compact(c.pools, c.d_table, c.d_lens, c.d_counts, workspace=big[8:])
    assert e.value.code == -9
    other = phs.PagedPool.empty(16, 4, 64)
    with pytest.raises(phs.PhsError) as e:
        phs.pages_compact([c.pools[0], other], c.d_table, c.d_lens, c.d_counts)
    assert e.value.code == -2
    c.check()
