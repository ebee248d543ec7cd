"""Refusals and host arithmetic of rotary positions, cache writes, the causal
convolution and the selective scan that need no GPU: every call here is refused
(or has nothing to do) before anything is launched."""
import ctypes
import math

import numpy as np
import pytest
import torch

import paged_hybrid_sliding_gb300 as phs
from paged_hybrid_sliding_gb300 import _lib

P = ctypes.c_void_p(1 << 20)   # an aligned address that no refused call reads
ODD = ctypes.c_void_p((1 << 20) + 8)
FAR = ctypes.c_void_p(1 << 24)


def ref(x):
    return None if x is None else ctypes.byref(x)


def paged(**kw):
    f = dict(k=P.value, v=P.value, num_pages=8, page_size=16, num_kv_heads=4, head_dim=64) | kw
    return _lib.PagedPoolC(*f.values())


def int8(**kw):
    f = dict(k=P.value, v=P.value, ks=P.value, vs=P.value, n=8, h=4, d=64) | kw
    return _lib.Int8PoolC(*f.values())


def rope(**kw):
    f = dict(turns=P.value, dim=64, interleaved=0, factor=1.0) | kw
    return _lib.RopeC(*f.values())


@pytest.mark.parametrize("change,code", [
    (dict(q=None), -1), (dict(q=ODD), -9), (dict(qs=128), -2), (dict(qs=257), -2),
    (dict(hq=0), -1), (dict(k=None), -1), (dict(ko=None), -1), (dict(ks=8), -2), (dict(hk=0), -1),
    (dict(d=96), -7), (dict(tokens=-1), -1), (dict(pos=None), -1), (dict(rope=None), -1),
    (dict(rope=rope(turns=0)), -1), (dict(rope=rope(dim=72)), -2), (dict(rope=rope(dim=24)), -7),
    (dict(rope=rope(factor=float("nan"))), -1), (dict(qo=ODD), -9), (dict(kos=60), -2),
    (dict(tokens=0), 0)])
def test_rope_rotate(change, code):
    a = dict(q=P, qs=256, hq=4, k=P, ks=128, hk=2, d=64, tokens=3, pos=P, rope=rope(), qo=P, qos=256,
             ko=P, kos=128) | change
    a["rope"] = ref(a["rope"])
    assert phs.lib().phs_rope_rotate(*a.values(), None) == code


@pytest.mark.parametrize("change,code", [
    (dict(pool=paged(head_dim=96)), -7), (dict(k=None), -1), (dict(v=ODD), -9), (dict(ks=8), -2),
    (dict(vs=260), -2), (dict(tokens=-1), -1), (dict(cu=None), -2), (dict(table=None), -1),
    (dict(width=0), -1), (dict(lens=None), -1), (dict(batch=-1), -1), (dict(rope=None), -1),
    (dict(rope=rope(dim=128)), -2), (dict(q=ODD), -9), (dict(qs=8), -2), (dict(hq=0), -1),
    (dict(qo=None), -1), (dict(i8=int8(h=2)), -2), (dict(i8=int8(d=128)), -2),
    (dict(i8=int8(ks=0)), -1), (dict(qt=None), -1), (dict(qb=None), -1), (dict(ql=None), -1),
    (dict(qw=0), -1), (dict(blocks=-1), -1), (dict(batch=70000), -7), (dict(batch=0), 0)])
def test_kv_write(change, code):
    a = dict(pool=paged(), k=P, ks=256, v=P, vs=256, tokens=9, cu=P, table=P, width=4, lens=P,
             batch=2, rope=rope(), q=P, qs=512, hq=8, qo=P, i8=int8(), qt=P, qw=4, qb=P, ql=P,
             blocks=3) | change
    for x in ("pool", "rope", "i8"):
        a[x] = ref(a[x])
    assert phs.lib().phs_kv_write_paged(*a.values(), None, None, None) == code


@pytest.mark.parametrize("change,code", [
    (dict(pool=paged(page_size=32)), -7), (dict(table=None), -1), (dict(starts=None), -1),
    (dict(cu=None), -1), (dict(width=0), -1), (dict(batch=-1), -1), (dict(tokens=-1), -1),
    (dict(most=-1), -1), (dict(batch=70000), -7), (dict(ko=None), -1), (dict(vo=ODD), -9),
    (dict(i8=int8(h=3)), -2), (dict(qt=None), -1), (dict(ql=None), -1), (dict(batch=0), 0)])
def test_kv_read(change, code):
    a = dict(pool=paged(), table=P, width=4, starts=P, cu=P, batch=2, tokens=9, most=9, i8=int8(),
             qt=P, qw=4, ql=P, ko=P, vo=P) | change
    for x in ("pool", "i8"):
        a[x] = ref(a[x])
    assert phs.lib().phs_kv_read_paged(*a.values(), None, None) == code


@pytest.mark.parametrize("change,code", [
    (dict(x=None), -1), (dict(x=ODD), -9), (dict(xs=56), -2), (dict(xs=68), -2),
    (dict(pool=dict(c=0)), -1), (dict(pool=dict(n=0)), -1), (dict(pool=dict(ch=60)), -7),
    (dict(pool=dict(w=1)), -7), (dict(pool=dict(w=5)), -7), (dict(weight=0), -1),
    (dict(weight=ODD.value), -9), (dict(bias=ODD.value), -9), (dict(batch=-1), -1),
    (dict(batch=9), -2), (dict(out=None), -1), (dict(batch=0), 0)])
def test_conv(change, code):
    a = dict(x=P, xs=64, weight=P.value, bias=0, batch=2, out=FAR, pool={}) | change
    pool = _lib.ConvPoolC(*(dict(c=P.value, n=4, ch=64, w=4) | a["pool"]).values())
    w = _lib.ConvWeightsC(a["weight"], a["bias"], 1)
    lib = phs.lib()
    assert lib.phs_causal_conv_prompt(a["x"], a["xs"], P, 9, ref(pool), ref(w), None, None,
                                      a["batch"], a["out"], None, None) == code
    if a["batch"] >= 0:
        assert lib.phs_causal_conv_decode(a["x"], a["xs"], ref(pool), ref(w), None, a["batch"],
                                          a["out"], None, None) == code
    assert lib.phs_causal_conv_prompt(P, 64, None, 9, ref(_lib.ConvPoolC(P.value, 4, 64, 4)),
                                      ref(_lib.ConvWeightsC(P.value, 0, 1)), None, None, 2, FAR, None,
                                      None) == -1


def test_conv_prompt_refuses_an_output_over_its_input():
    pool, w = _lib.ConvPoolC(P.value, 4, 64, 4), _lib.ConvWeightsC(P.value, 0, 1)
    for out in (1 << 20, (1 << 20) + 9 * 128 - 16, (1 << 20) - 9 * 128 + 16):
        assert phs.lib().phs_causal_conv_prompt(P, 64, P, 9, ref(pool), ref(w), None, None, 2,
                                                ctypes.c_void_p(out), None, None) == -1
    assert phs.lib().phs_causal_conv_prompt(P, 64, P, 9, ref(pool), ref(w), None, None, 0,
                                            ctypes.c_void_p((1 << 20) + 9 * 128), None, None) == 0


def at(address):
    return ctypes.c_void_p(address)


BASE = 1 << 20


def test_more_rows_than_a_tile_counts():
    pool, w = _lib.ConvPoolC(P.value, 4, 64, 4), _lib.ConvWeightsC(P.value, 0, 1)
    assert phs.lib().phs_causal_conv_prompt(P, 64, P, 2**31 - 9, ref(pool), ref(w), None, None, 2,
                                            at(1 << 50), None, None) == -7


@pytest.mark.parametrize("q,qs,k,ks,qo,qos,ko,kos", [
    # (9 tokens of 4 and 2 heads of 64: 512 and 256 bytes a row)
    (0, 256, 1 << 20, 128, 16, 256, 2 << 20, 128),            # q_out over q, 16 bytes on
    (0, 384, 1 << 20, 128, 0, 256, 2 << 20, 128),             # another stride
    (0, 256, 1 << 20, 128, 2 << 20, 256, (1 << 20) + 9 * 256 - 16, 128),  # k_out over k's last
    (0, 256, 1 << 20, 128, 1 << 20, 256, 2 << 20, 128),       # q_out over k
    (0, 256, 1 << 20, 128, 2 << 20, 256, 8 * 512, 128),       # k_out over q
    (0, 384, 512, 384, 2 << 20, 384, (2 << 20) + 496, 384),   # k_out over q_out in one row
    (0, 384, 512, 384, 2 << 20, 384, (2 << 20) + 528, 384)])  # ... and in the next row
def test_rotate_refuses_outputs_over_others(q, qs, k, ks, qo, qos, ko, kos):
    a = [at(BASE + q), qs, 4, at(BASE + k), ks, 2, 64, 9, P, ref(rope()), at(BASE + qo), qos,
         at(BASE + ko), kos, None]
    assert phs.lib().phs_rope_rotate(*a) == -1


@pytest.mark.parametrize("q,qs,k,v,qo", [
    (0, 512, 1 << 20, 2 << 20, 16), (0, 768, 1 << 20, 2 << 20, 0),
    (0, 512, 1 << 20, 2 << 20, (1 << 20) + 9 * 512 - 16),
    (0, 512, 1 << 20, 2 << 20, (2 << 20) - 9 * 1024 + 16)])
def test_write_refuses_an_output_over_its_inputs(q, qs, k, v, qo):
    a = [ref(paged()), at(BASE + k), 256, at(BASE + v), 256, 9, P, P, 4, P, 2, ref(rope()),
         at(BASE + q), qs, 8, at(BASE + qo)]
    assert phs.lib().phs_kv_write_paged(*a, None, None, 0, None, None, 0, None, None, None) == -1


@pytest.mark.parametrize("out,stride", [(16, 64), (-16, 64), (0, 72), (2 * 72 * 2 - 16, 72)])
def test_conv_of_a_token_refuses_an_output_over_a_part_of_its_input(out, stride):
    pool, w = _lib.ConvPoolC(P.value, 4, 64, 4), _lib.ConvWeightsC(P.value, 0, 1)
    assert phs.lib().phs_causal_conv_decode(P, stride, ref(pool), ref(w), None, 3, at(BASE + out),
                                            None, None) == -1


@pytest.mark.parametrize("over", ["x", "b", "c", "dt"])
def test_scan_refuses_an_output_over_its_inputs(over):
    where = dict(x=0, b=1 << 20, c=2 << 20, dt=3 << 20)
    v = {n: BASE + d for n, d in where.items()}
    inputs = _lib.ScanInputsC(v["x"], v["b"], v["c"], v["dt"], 256, 128, 128, 4, 2, 0)
    pool, w = _lib.ScanPoolC(P.value, 4, 4, 64, 64), _lib.ScanWeightsC(P.value, 0, 0)
    lib = phs.lib()
    assert lib.phs_selective_scan_decode(ref(inputs), ref(pool), ref(w), None, 2, at(v[over]), 1,
                                         None, None) == -1
    # its last bytes over the first ones
    assert lib.phs_selective_scan_decode(ref(inputs), ref(pool), ref(w), None, 2,
                                         at(v[over] - 2 * 1024 + 16), 1, None, None) == -1


@pytest.mark.parametrize("change,code", [
    (dict(x=0), -1), (dict(x=ODD.value), -9), (dict(b=0), -1), (dict(c=ODD.value), -9),
    (dict(dt=0), -1), (dict(xs=128), -2), (dict(xs=260), -2), (dict(bs=64), -2), (dict(cs=64), -2),
    (dict(ds=3), -2), (dict(g=0), -1), (dict(g=3), -2), (dict(kind=2), -1),
    (dict(pool=dict(s=0)), -1), (dict(pool=dict(s=ODD.value)), -9), (dict(pool=dict(p=96)), -7),
    (dict(pool=dict(n=32)), -7), (dict(pool=dict(h=0)), -1), (dict(rate=0), -1),
    (dict(batch=-1), -1), (dict(batch=9), -2), (dict(out=None), -1), (dict(batch=0), 0)])
def test_scan(change, code):
    a = dict(x=P.value, b=P.value, c=P.value, dt=P.value, xs=256, bs=128, cs=128, ds=4, g=2, kind=0,
             pool={}, rate=P.value, batch=2, out=P) | change
    inputs = _lib.ScanInputsC(*[a[n] for n in ("x", "b", "c", "dt", "xs", "bs", "cs", "ds", "g",
                                               "kind")])
    pool = _lib.ScanPoolC(*(dict(s=P.value, k=4, h=4, p=64, n=64) | a["pool"]).values())
    w = _lib.ScanWeightsC(a["rate"], 0, 0)
    lib = phs.lib()
    assert lib.phs_selective_scan_prompt(ref(inputs), P, 100, 64, ref(pool), ref(w), None, None,
                                         a["batch"], a["out"], P, 1 << 26, None, None) == code
    if a["batch"] >= 0:
        assert lib.phs_selective_scan_decode(ref(inputs), ref(pool), ref(w), None, a["batch"],
                                             a["out"], 1, None, None) == code


@pytest.mark.parametrize("change,code", [
    (dict(cu=None), -1), (dict(tokens=-1), -1), (dict(most=-1), -1), (dict(ws=None), -5),
    (dict(ws=ODD), -9)])
def test_scan_prompt(change, code):
    a = dict(cu=P, tokens=100, most=64, ws=P) | change
    v = P.value
    assert phs.lib().phs_selective_scan_prompt(
        ref(_lib.ScanInputsC(v, v, v, v, 256, 128, 128, 4, 2, 0)), a["cu"], a["tokens"], a["most"],
        ref(_lib.ScanPoolC(v, 4, 4, 64, 64)), ref(_lib.ScanWeightsC(v, 0, 0)), None, None, 2, P,
        a["ws"], 1 << 26, None, None) == code


def test_workspace_sizes():
    assert phs.scan_prompt_workspace_bytes(1, 3, 2, 64, 64, 10, 10) == 0
    assert phs.scan_prompt_workspace_bytes(1, 2, 2, 96, 64, 10, 10) == 0
    assert phs.scan_prompt_workspace_bytes(1, 2, 2, 64, 32, 10, 10) == 0
    assert phs.scan_prompt_workspace_bytes(-1, 2, 2, 64, 64, 10, 10) == 0


def test_binding_wants_cuda_tensors():
    x = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        phs.kv_write_paged(phs.PagedPool.empty(2, 4, 64, device="cpu"), x, x, i[None], i)
    with pytest.raises(ValueError):
        phs.rope_rotate(x, None, i, phs.Rope.make(64, device="cpu"))
    with pytest.raises(ValueError):
        phs.causal_conv_decode(x[0], phs.ConvPool.zeros(2, 64, 4, device="cpu"),
                               phs.ConvWeights(torch.zeros(64, 4)))
    with pytest.raises(ValueError):
        phs.selective_scan_decode(x, x[..., 0], x, x, phs.ScanPool.zeros(2, 4, 64, 64, "cpu"),
                                  phs.ScanWeights(torch.zeros(4)))


# ------------------------------------------------------------ frequencies --
def test_turns_are_the_frequencies():
    r = phs.Rope.make(64, base=500.0, device="cpu")
    f = phs.rope_frequencies(64, base=500.0)[0]
    assert r.turns.shape == (32,) and r.factor == 1.0 and not r.interleaved
    got = r.turns.numpy().view(np.uint64).astype(np.float64) / 2.0 ** 64 * 2 * math.pi
    assert np.allclose(got, f, rtol=1e-15, atol=0)
    assert np.allclose(f, [500.0 ** (-i / 32) for i in range(32)], rtol=1e-14)


def test_an_angle_of_a_far_position_is_exact():
    """position * turns modulo 2^64 against the angle in rational arithmetic."""
    from fractions import Fraction
    r = phs.Rope.make(16, base=10000.0, device="cpu")
    for t in r.turns.tolist():
        t %= 2 ** 64
        for pos in (1, 4095, 250_001, 2 ** 31 - 1):
            want = Fraction(t * pos, 2 ** 64) % 1
            assert Fraction((t * pos) % 2 ** 64, 2 ** 64) == want


def test_scalings():
    plain = phs.rope_frequencies(128)[0]
    f, m = phs.rope_frequencies(128, scaling="linear", scale=4.0)
    assert np.allclose(f, plain / 4) and m == 1.0
    f, m = phs.rope_frequencies(128, scaling="base", scale=4.0)
    assert f[0] == plain[0] and math.isclose(f[-1], plain[-1] / 4, rel_tol=1e-12) and m == 1.0
    for kind, high, mag in (("parts", 32, 0.1 * math.log(8) + 1), ("wavelengths", 4, 1.0)):
        f, m = phs.rope_frequencies(128, scaling=kind, scale=8.0, trained_len=4096)
        turns = 4096 * plain / (2 * math.pi)
        assert math.isclose(m, mag)
        assert np.all(np.diff(f) < 0) and np.all(f <= plain) and np.all(f >= plain / 8 * (1 - 1e-12))
        # one pair's margin: `parts` rounds the ramp's ends to whole pairs
        step = 10000.0 ** (1 / 64)
        assert np.allclose(f[turns > high * step], plain[turns > high * step])
        assert np.allclose(f[turns < 1 / step], plain[turns < 1 / step] / 8)
        mid = (turns < high / step) & (turns > step)
        assert np.all(f[mid] < plain[mid]) and np.all(f[mid] > plain[mid] / 8)


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=15), dict(rotary_dim=0), dict(rotary_dim=64, base=1.0),
    dict(rotary_dim=64, scaling="other"), dict(rotary_dim=64, scaling="linear", scale=0.5),
    dict(rotary_dim=64, scaling="parts", scale=2.0),
    dict(rotary_dim=64, scaling="wavelengths", scale=2.0, trained_len=4096, low=4, high=4),
    dict(rotary_dim=2, scaling="base", scale=2.0)])
def test_scalings_refused(kw):
    with pytest.raises(ValueError):
        phs.Rope.make(**kw, device="cpu")
