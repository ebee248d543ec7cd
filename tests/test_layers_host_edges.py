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


# --------------------------------------------------------- 32-bit row counts --
# (a kernel's last tile ends behind the last token: its rows must not pass 2^31)
MANY = 2 ** 31 - 9


def ref(x):
    return ctypes.byref(x)


def pool(**kw):
    return phs._lib.PagedPoolC(P.value, P.value, 8, 16, kw.get("heads", 1), 64)


ROPE = phs._lib.RopeC(P.value, 64, 0, 1.0)


@pytest.mark.parametrize("tokens,q_heads,k_heads", [(MANY, 1, 1), (3, 2 ** 25, 1), (3, 1, 2 ** 25)])
def test_rotate_refuses_rows_past_32_bits(tokens, q_heads, k_heads):
    qs, ks = q_heads * 64, k_heads * 64
    assert phs.lib().phs_rope_rotate(P, qs, q_heads, FAR, ks, k_heads, 64, tokens, P, ref(ROPE), P,
                                     qs, FAR, ks, None) == -7


@pytest.mark.parametrize("tokens,q_heads", [(MANY, 1), (3, 2 ** 25)])
def test_write_refuses_rows_past_32_bits(tokens, q_heads):
    far = [ctypes.c_void_p(i << 50) for i in (1, 2, 3)]
    assert phs.lib().phs_kv_write_paged(ref(pool()), far[0], 64, far[1], 64, tokens, P, P, 4, P, 2,
                                        ref(ROPE), P, q_heads * 64, q_heads, far[2], None, None, 0,
                                        None, None, 0, None, None, None) == -7


def test_read_refuses_rows_past_32_bits():
    assert phs.lib().phs_kv_read_paged(ref(pool()), P, 4, P, P, 2, MANY, MANY, None, None, 0, None, P,
                                       FAR, None, None) == -7


def test_scan_refuses_rows_past_32_bits():
    v = [i << 50 for i in (1, 2, 3, 4)]
    inputs = phs._lib.ScanInputsC(*v, 64, 64, 64, 1, 1, 0)
    assert phs.lib().phs_selective_scan_prompt(
        ref(inputs), P, MANY, MANY, ref(phs._lib.ScanPoolC(P.value, 4, 1, 64, 64)),
        ref(phs._lib.ScanWeightsC(P.value, 0, 0)), None, None, 2, ctypes.c_void_p(5 << 50), P, 2 ** 62,
        None, None) == -7


# --------------------------------------------------------------- workspaces --
@pytest.mark.parametrize("B,total,most", [(256, 1024, 4), (65535, 65535 * 16, 16), (1, 0, 0),
                                          (3, 16, 400), (0, 0, 0)])
def test_scans_token_by_token_need_next_to_no_workspace(B, total, most):
    """Calls whose requests all go token by token keep nothing in the workspace;
    0 stays the answer for what is not supported."""
    assert phs.scan_prompt_workspace_bytes(B, 64, 8, 64, 128, total, most) == 256
    assert phs.scan_prompt_workspace_bytes(B, 64, 8, 96, 128, total, most) == 0
    assert phs.scan_prompt_workspace_bytes(B, 65536, 8, 64, 128, total, most) == 0


# ------------------------------------------------------ longest requests first --
def by_length(cu, at, short_len):
    """The scan's choice of the request that comes `at`-th, its threads one
    after another: every request that may be written as the answer."""
    B = len(cu) - 1
    lens = [cu[j + 1] - cu[j] for j in range(B)]
    more = [n > short_len for n in lens]
    if at >= sum(more):
        return [j for j in range(B) if not more[j]]
    return [j for j in range(B) if more[j] and
            sum(lens[i] > lens[j] or (lens[i] == lens[j] and i < j) for i in range(B)) == at]


def test_longest_first_is_a_permutation():
    """Whatever the offsets (falling ones among them), each place of a call gets
    a request: the longer ones one place each, longest first, the others' places
    any short one."""
    rng = np.random.default_rng(1)
    for trial in range(300):
        B = int(rng.integers(2, 40))
        kind = trial % 3
        if kind == 0:
            cu = np.concatenate([[0], np.cumsum(rng.integers(0, 40, B))])
        elif kind == 1:
            cu = np.concatenate([[0], np.cumsum(rng.choice([0, 5, 16, 17, 300], B))])
        else:
            cu = rng.integers(-50, 500, B + 1)
        cu = cu.tolist()
        lens = [cu[j + 1] - cu[j] for j in range(B)]
        longer = [j for j in range(B) if lens[j] > 16]
        got = [by_length(cu, at, 16) for at in range(B)]
        assert all(len(g) == 1 for g in got[:len(longer)])
        order = [g[0] for g in got[:len(longer)]]
        assert sorted(order) == longer
        assert order == sorted(longer, key=lambda j: (-lens[j], j))
        assert all(g and all(lens[j] <= 16 for j in g) for g in got[len(longer):])


# ------------------------------------------------------------------- angles --
def test_turns_against_angles_of_60_digits():
    """The angle that position * turns (modulo 2^64) stands for, against base^(-2 i /
    rotary_dim) * position / 2 pi in 60 decimal digits.  Frequencies are fp64:
    a power, a product and a quotient, 2^-50 of themselves; turns round by
    2^-65 of a turn; each a position's times."""
    from decimal import Decimal, getcontext
    getcontext().prec = 60

    def arctan_inverse(n):                       # of 1 / n
        total, term, k = Decimal(0), Decimal(1) / n, 0
        while abs(term) > Decimal(10) ** -58:
            total += term / (2 * k + 1) * (-1) ** k
            term, k = term / (n * n), k + 1
        return total

    pi = 4 * (4 * arctan_inverse(5) - arctan_inverse(239))
    for dim, base in ((16, 10000.0), (64, 500.0), (128, 1e6)):
        turns = phs.Rope.make(dim, base=base, device="cpu").turns.numpy().view(np.uint64).tolist()
        for i, t in enumerate(turns):
            turn = Decimal(base) ** (Decimal(-2 * i) / dim) / (2 * pi)
            for pos in (1, 4095, 250_001, 2 ** 31 - 1):
                got = Decimal((t * pos) % 2 ** 64) / 2 ** 64
                off = (got - turn * pos) % 1     # of a turn, either way round
                off = min(abs(off), 1 - abs(off))
                assert off <= pos * (Decimal(2) ** -65 + turn * Decimal(2) ** -50), (dim, i, pos)
