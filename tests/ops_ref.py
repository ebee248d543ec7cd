"""64-bit reference forms of the page operations, differential attention and
linear attention: plain loops over the definitions, and the error bounds
that the GPU tests hold the kernels to."""
from __future__ import annotations

import math

import numpy as np
import torch

PAGE = 16


# ------------------------------------------------------------------- pages --
def pages(n):
    return (int(n) + PAGE - 1) // PAGE


def free_rows(table, lens, counts, rows):
    for r in rows:
        for j in range(pages(lens[r])):
            counts[table[r, j]] -= 1
        lens[r] = 0


def fork_rows(pools, table, lens, counts, src, dst):
    """pools: list of (k, v) arrays, changed in place like the rest."""
    free = [p for p in range(len(counts)) if counts[p] == 0]
    for s, d in zip(src, dst):
        for j in range(pages(lens[s])):
            p = table[s, j]
            if (j + 1) * PAGE > lens[s]:
                new = free.pop(0)
                for k, v in pools:
                    k[new], v[new] = k[p].copy(), v[p].copy()
                p = new
            table[d, j] = p
            counts[p] += 1
        lens[d] = lens[s]


def compact(pools, table, lens, counts):
    """Returns (page_map, live)."""
    live = int((counts > 0).sum())
    highs = [p for p in range(len(counts) - 1, live - 1, -1) if counts[p] > 0]
    lows = [p for p in range(live) if counts[p] <= 0]
    page_map = np.where(counts > 0, np.arange(len(counts)), -1).astype(np.int32)
    for a, b in zip(highs, lows):
        page_map[a] = b
        counts[b], counts[a] = counts[a], 0
        for k, v in pools:
            k[b], v[b] = k[a].copy(), v[a].copy()
    for r in range(len(lens)):
        for j in range(pages(lens[r])):
            table[r, j] = page_map[table[r, j]]
    return page_map, live


# --------------------------------------------------- differential attention --
def diff_decode(q, k, v, table, lens, lam_vecs, lam_init, norm, eps, scale, out_eps):
    """(out, bound), both [B, H, 2D] fp64.  q, k, v bf16 tensors, table and
    lens host arrays.  out_eps: half a step of the output type.

    Bound, from the formula: a score is D products summed in fp32, off by at
    most D 2^-24 of its absolute sum, and with its scaling and exponential
    (2 ulp) a weight is off by delta = 2 (D 2^-24 max|s| + 2^-22) relative.
    Weights of the value product are held to 16 bits or more (2^-16 of each
    weight), and n of them are summed in fp32 (n 2^-24).  Both maps' terms
    add up: rel (p1 |v| + |lambda| p2 |v|), rel = 2 delta + 2^-16 + n 2^-23;
    lambda, the norm and the final products add 2^-20 of the result.  The norm
    divides by a root mean square that is off by at most the bound's own."""
    B, H2, D = q.shape
    H, Hv = H2 // 2, k.shape[1] // 2
    G = H // Hv
    q, dev = q.double(), q.device
    out = torch.zeros((B, H, 2 * D), dtype=torch.float64, device=dev)
    bound = torch.zeros_like(out)
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            continue
        ids = torch.from_numpy(np.ascontiguousarray(table[b, :pages(n)]).astype(np.int64)).to(dev)
        kb = k[ids].double().transpose(0, 1).reshape(2 * Hv, -1, D)[:, :n]
        vb = v[ids].double().transpose(0, 1).reshape(2 * Hv, -1, D)[:, :n]
        for i in range(H):
            j = i // G
            lam = (torch.exp((lam_vecs[0].double() * lam_vecs[1].double()).reshape(-1, D)
                             [min(i, lam_vecs[0].numel() // D - 1)].sum())
                   - torch.exp((lam_vecs[2].double() * lam_vecs[3].double()).reshape(-1, D)
                               [min(i, lam_vecs[0].numel() // D - 1)].sum()) + lam_init)
            vj = torch.cat([vb[2 * j], vb[2 * j + 1]], 1)
            x = torch.zeros(2 * D, dtype=torch.float64, device=dev)
            e = torch.zeros_like(x)
            for m in (0, 1):
                s = kb[2 * j + m] @ q[b, 2 * i + m] * scale
                top = float((kb[2 * j + m].abs() @ q[b, 2 * i + m].abs() * scale).max())
                p = torch.softmax(s, 0)
                rel = 4 * (D * 2**-24 * top + 2**-22) + 2**-16 + n * 2**-23
                w = 1.0 if m == 0 else -lam
                x = x + w * (p @ vj)
                e = e + abs(w) * rel * (p @ vj.abs())
            e = e + 2**-20 * x.abs()
            if norm is not None:
                r = torch.sqrt((x @ x) / (2 * D) + eps)
                g = norm.double() * (1 - lam_init)
                e = (g.abs() / r) * (e + x.abs() * (e.norm() / math.sqrt(2 * D) / r)) * 1.01
                x = x / r * g
                e = e + 2**-20 * x.abs()
            out[b, i] = x
            bound[b, i] = e + out_eps * x.abs()
    return out, bound


# --------------------------------------------------------- linear attention --
def linear(q, k, v, state, decay_log, scale):
    """The recurrence over the tokens of one request, and over the absolute
    values of everything: (out [T, Hq, D], state, |out| sums, |state| sums),
    fp64.  q [T, Hq, D], k, v [T, Hkv, D], state [Hkv, D, D]."""
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    g = torch.exp(decay_log.double())[:, None, None]
    S, A = state.double(), state.double().abs()
    qd = q.double().view(T, Hkv, Hq // Hkv, D) * scale
    kd, vd = k.double(), v.double()
    out, mag = [], []
    for t in range(T):
        kv = kd[t, :, :, None] * vd[t, :, None, :]
        S = S * g + kv
        A = A * g + kv.abs()
        out.append((qd[t] @ S).reshape(Hq, D))
        mag.append((qd[t].abs() @ A).reshape(Hq, D))
    if not out:
        e = torch.zeros((0, Hq, D), dtype=torch.float64, device=q.device)
        return e, S, e, A
    return torch.stack(out), S, torch.stack(mag), A
