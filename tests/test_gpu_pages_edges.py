"""Page operations with table entries that name no live page."""
import numpy as np
import pytest

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
