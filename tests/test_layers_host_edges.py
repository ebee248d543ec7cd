"""Host arithmetic and refusals of rotary positions, cache writes and the scan
at sizes and lengths that ordinary calls stay away from; no GPU."""
import ctypes
import math

import numpy as np
import pytest

import paged_hybrid_sliding_gb300 as phs

P = ctypes.c_void_p(1 << 20)   # an aligned address that no refused call reads
FAR = ctypes.c_void_p(1 << 50)


# ------------------------------------------------------------ frequencies --
@pytest.mark.parametrize("dim,base,trained", [(128, 10000.0, 131072), (64, 10000.0, 262144),
                                              (32, 500.0, 32768)])
def test_parts_where_every_pair_turns_more_than_once(dim, base, trained):
    """A trained length in which even the slowest pair makes more than `low`
    rotations: it is still between the two ends, not `scale` times slower."""
    plain = phs.rope_frequencies(dim, base)[0]
    turns = trained * plain / (2 * math.pi)
    assert turns[-1] > 1.5
    f, _ = phs.rope_frequencies(dim, base, scaling="parts", scale=8.0, trained_len=trained)
    # by the index: from the last whole pair of 32 rotations to the first of one
    at = [dim / 2 * math.log(trained / (2 * math.pi * r)) / math.log(base) for r in (32, 1)]
    slow = np.clip((np.arange(dim // 2) - math.floor(at[0])) / (math.ceil(at[1]) - math.floor(at[0])),
                   0, 1)
    assert np.allclose(f, plain * (1 - slow) + plain / 8 * slow, rtol=1e-13, atol=0)
    assert plain[-1] / 8 * 1.05 < f[-1] < plain[-1]
