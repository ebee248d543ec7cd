"""64-bit reference forms of rotary positions, the 8-bit cache form, the causal
convolution and the selective scan: plain loops over the definitions, and the
error bounds that the GPU tests hold the kernels to."""
from __future__ import annotations

import math

import numpy as np
import torch

PAGE, QBLOCK = 16, 32


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


# ------------------------------------------------------------------- rotary --
def rotated(x, positions, freq, interleaved, factor):
    """(y, bound) of x [T, H, D] (bf16) turned by positions[t] * freq radians.

    Bound: the angle is held to 32 bits of a turn and rounded to 24 bits of
    half a turn (pi 2^-25), sine and cosine to 2 ulp (2^-23), factor, product
    and sum to 2^-24 each, at most 2^-20 of factor (|a| + |b|) in all; and half
    a step of bf16."""
    r = 2 * len(freq)
    angle = positions.double()[:, None] * torch.as_tensor(freq, device=x.device)
    cos, sin = (torch.cos(angle) * factor)[:, None], (torch.sin(angle) * factor)[:, None]
    y = x.double().clone()
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else \
        (x[..., :r // 2], x[..., r // 2:r])
    a, b = a.double(), b.double()
    bound = torch.zeros_like(y)
    e = (a.abs() + b.abs()) * abs(factor) * 2.0 ** -20
    u, v = a * cos - b * sin, b * cos + a * sin
    for part, val in ((0, u), (1, v)):
        at = (slice(part, r, 2) if interleaved else slice(part * r // 2, (part + 1) * r // 2))
        y[..., at] = val
        bound[..., at] = e + val.abs() * half_step(torch.bfloat16)
    return y, bound


# ----------------------------------------------------------------- 8 bits --
def quantise(x):
    """(codes int8, scale fp32) of one block [32, D] of bf16 values, in IEEE
    single precision."""
    x = x.float().cpu().numpy()
    s = np.float32(np.abs(x).max()) / np.float32(127)
    if s == 0:
        return np.zeros(x.shape, np.int8), s
    return np.clip(np.rint(x / s), -127, 127).astype(np.int8), s


# -------------------------------------------------------------- convolution --
def conv(x, old, weight, bias, silu):
    """(y, bound, last inputs) of one request: x [T, C] behind old [W - 1, C].

    Bound: W products and sums in fp32, 2 W 2^-24 of the absolute sum, which
    the activation passes on with a slope below 1.1; its exponential is off by
    the argument's rounding (2^-23 |y|) and 2^-22, its quotient by 2^-22, of a
    result below |y|; below -87 the true result is under 2^-117 and may come
    out as zero; and half a step of bf16."""
    W = weight.shape[1]
    z = torch.cat([old.double(), x.double()])
    w, T = weight.double(), x.shape[0]
    y = torch.zeros((T, x.shape[1]), dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(y)
    if bias is not None:
        y, mag = y + bias.double(), mag + bias.double().abs()
    for k in range(W):
        y = y + z[k:k + T] * w[:, k]
        mag = mag + (z[k:k + T] * w[:, k]).abs()
    e = (2 * W + 2) * 2.0 ** -24 * mag
    if silu:
        s = y * torch.sigmoid(y)
        e = 1.1 * e + s.abs() * ((y.abs() + e) * 2.0 ** -23 + 2.0 ** -20) + 2.0 ** -117
        y = s
    return y, e + y.abs() * half_step(torch.bfloat16), z[T:].to(x.dtype)


# --------------------------------------------------------------------- scan --
def softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))


def scan(x, dt, b, c, state, rate, skip, dt_bias):
    """The recurrence over the tokens of one request, and over the absolute
    values of everything: (out [T, H, P], state, |out| sums, |state| sums, log
    decays [T, H]), fp64."""
    T, H, P = x.shape
    g = H // b.shape[1]
    s = dt.double() if dt_bias is None else dt.double() + dt_bias.double()
    s = softplus(s)
    log = s * rate.double()
    S, A = state.double(), state.double().abs()
    xd, bd = x.double(), b.double().repeat_interleave(g, 1)
    cd = c.double().repeat_interleave(g, 1)
    out, mag = [], []
    for t in range(T):
        f = torch.exp(log[t])[:, None, None]
        add = (s[t][:, None] * xd[t])[..., None] * bd[t][:, None]
        S, A = S * f + add, A * f + add.abs()
        y, m = (S @ cd[t][..., None])[..., 0], (A @ cd[t].abs()[..., None])[..., 0]
        if skip is not None:
            y, m = y + skip.double()[:, None] * xd[t], m + (skip.double()[:, None] * xd[t]).abs()
        out.append(y)
        mag.append(m)
    if not out:
        e = torch.zeros((0, H, P), dtype=torch.float64, device=x.device)
        return e, S, e, A, log
    return torch.stack(out), S, torch.stack(mag), A, log


def scan_bounds(ref, mag, smag, log, out_dtype, N, chunked):
    """(bound of out, bound of the state).

    One token at a time: decay, product and sum round by 2^-24 each and the
    decay factor is off by 2^-22 and by its argument's error, the step's 2^-22
    of it: with T tokens (T + 8) 2^-22 of the absolute sums, and (1 + max |log
    decay|) times that.  Chunks of 128 sum the log decays: a sum is off by 16
    roundings of 2^-24 of the chunk's absolute sum X, a difference of two by
    twice that, which is what its exponential is off by, and as many for each
    chunk; steps are off by 2^-22.  Products of an output hold the weights of a
    chunk's own tokens and the state before it to bf16 (half a step, 2^-8 of
    each), a state's products hold 24 bits."""
    T = log.shape[0]
    big = float(log.abs().max()) if T else 0.0
    rel = (T + 8) * 2.0 ** -22 * (1 + big)
    if chunked and T:
        X = max(float(log[i:i + 128].abs().sum(0).max()) for i in range(0, T, 128))
        rel = rel + (T // 128 + 1) * 2.0 ** -19 * X
    soft = 2.0 ** -8 if chunked else 0.0
    return mag * (rel + N * 2.0 ** -23 + soft) + ref.abs() * half_step(out_dtype), smag * rel


def close(got, ref, bound, what):
    err = (got.double() - ref).abs()
    assert torch.isfinite(got).all(), what
    assert bool((err <= bound).all()), \
        f"{what}: err {float(err.max()):.3e}, worst excess {float((err - bound).max()):.3e}"
