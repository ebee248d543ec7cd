"""Page operations with table entries that name no live page, and over more
than one tile of ids and of entries."""
import numpy as np
import pytest
import torch

import ops_ref
import paged_hybrid_sliding_gb300 as phs
from gpu_util import dev
from test_gpu_pages import Cache

pytestmark = pytest.mark.gpu


def test_fork_does_not_share_a_page_that_it_has_just_given_out():
    """A whole page's entry that names a free page is no reference to a live
    page, also where the same call takes that page as a fresh one."""
    c = Cache([40, 20, 0, 0], 16, 25)
    free = np.flatnonzero(c.counts == 0)
    c.table[0, 0] = free[0]          # 40 tokens: entries 0 and 1 are whole pages
    c.table[1, 0] = free[1]
    c.d_table.copy_(dev(c.table))
    c.fork([0, 1], [2, 3], host=False)
    c.counts[c.table[0, 1]] += 1     # the one good whole page
    c.counts[free[:2]] = 1           # the two fresh pages: one row each
    c.table[2, :3] = [free[0], c.table[0, 1], free[0]]
    c.table[3, :2] = [free[1], free[1]]
    c.lens[2:] = [40, 20]
    for src, dst in ((c.table[0, 2], free[0]), (c.table[1, 1], free[1])):
        for k, v in c.host:
            k[dst], v[dst] = k[src].copy(), v[src].copy()
    c.check(-3)


@pytest.mark.parametrize("children", [1, 31, 300])
def test_fork_from_rows_with_dead_entries_among_many_fresh_pages(children):
    """Entries of dead pages anywhere among the fresh ones, and behind them."""
    rs = np.random.RandomState(children)
    c = Cache([200] + [0] * children, 700, 27, layers=1, heads=1)
    free = np.flatnonzero(c.counts == 0)
    dead = [free[0], free[children - 1], free[children], free[-1], free[rs.randint(children)]]
    at = [0, 3, 5, 6, 11]            # of the row's 12 whole pages
    c.table[0, at] = dead
    c.d_table.copy_(dev(c.table))
    order = rs.permutation(children) + 1
    c.fork([0] * children, list(order), host=False)
    for i, d in enumerate(order):
        c.table[d, :12] = c.table[0, :12]
        c.table[d, 12] = free[i]
        c.lens[d] = 200
        for k, v in c.host:
            k[free[i]], v[free[i]] = k[c.table[0, 12]].copy(), v[c.table[0, 12]].copy()
    live = [j for j in range(12) if j not in at]
    c.counts[c.table[0, live]] += children
    c.counts[free[:children]] = 1
    c.check(-3)


def test_fork_of_more_entries_than_a_tile():
    """8,500 entries, of which every third needs no page: the ranks of fresh
    pages go on from tile to tile."""
    n = 8500
    lens = [16 if r % 3 == 0 else 1 + r % 15 for r in range(n)] + [0] * n
    c = Cache(lens, 20_000, 29, layers=1, heads=1, width=1)
    rs = np.random.RandomState(2)
    c.fork(list(rs.permutation(n)), [n + r for r in rs.permutation(n)])
    c.check()


@pytest.mark.parametrize("below", [0, 1, 40, 8191])
def test_fresh_pages_on_both_sides_of_a_tile(below):
    """All but `below` of the first 8,192 pages are taken: the search goes on in
    the next tiles."""
    n, pages = 60, 25_000
    c = Cache([5] * n + [0] * n, pages, 31, layers=1, heads=1, width=1)
    rs = np.random.RandomState(below)
    c.counts[:8192][c.counts[:8192] == 0] = 1           # held by nobody's row
    c.counts[8192:16_384] += 1                          # and the second tile is full
    spare = [p for p in rs.permutation(8192) if p not in set(c.table[:n, 0])][:below]
    c.counts[spare] = 0
    c.d_counts.copy_(dev(c.counts))
    c.fork(list(range(n)), list(range(n, 2 * n)))
    c.check()


@pytest.mark.parametrize("num_pages", [8191, 8192, 8193, 16_384, 20_001])
@pytest.mark.parametrize("share", [0.03, 0.5, 0.99])
def test_compact_over_tiles(num_pages, share):
    """Live pages anywhere among all ids, every map entry, count, table cell and
    page checked."""
    lens = [16 * max(1, int(num_pages * share / 8)) - 3] * 8
    c = Cache(lens, num_pages, 33, layers=1, heads=1, shared=1)
    page_map, live = phs.pages_compact(c.pools, c.d_table, c.d_lens, c.d_counts, status=c.status)
    ref_map, ref_live = ops_ref.compact(c.host, c.table, c.lens, c.counts)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(page_map.cpu().numpy(), ref_map)
    assert int(live.item()) == ref_live
    c.check()
