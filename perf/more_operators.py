"""Measured cases of what the layers of a hybrid serving stack do with their tokens beside attention:

  write   rotary positions of queries and keys as the tokens enter the paged cache, for whole
          prompts (ragged, packed) and for one new token per request
  write8  the same into a cache whose older blocks of 32 tokens are held in 8 bits, quantised as
          they are written, and the written tokens read back
  conv    the short causal convolution of a selective state space layer
  scan    the selective scan behind it: states that decay by each token's own step, for whole
          prompts and for one new token per request

`run` computes them in plain torch where `own` is false and through the package's entry points
where it is true.
"""
import math

import numpy as np
import torch

own = False

PAGE, BLOCK = 16, 32
DEV = "cuda"


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # one token of two short conversations of a two-layer stack: latency
        dict(name="write_2req_token", op="write", batch=2, lo=1, hi=1, ctx_lo=37, ctx_hi=200,
             q_heads=4, kv_heads=2, dim=64, rotary=64, pairs="halves", scaling="none"),
        # one token of a full serving batch, half of each head rotated
        dict(name="write_256req_token", op="write", batch=256, lo=1, hi=1, ctx_lo=100, ctx_hi=2000,
             q_heads=32, kv_heads=8, dim=128, rotary=64, pairs="neighbours", scaling="linear"),
        # one long prompt, positions scaled for long contexts
        dict(name="write_1req_32k", op="write", batch=1, lo=32751, hi=32751, ctx_lo=0, ctx_hi=0,
             q_heads=32, kv_heads=8, dim=128, rotary=128, pairs="halves", scaling="parts"),
        # a batch of short parts of prompts whose earlier tokens are cached in 8 bits
        dict(name="write8_16req_short", op="write8", batch=16, lo=1, hi=517, ctx_lo=5, ctx_hi=4000,
             hot=64, q_heads=32, kv_heads=8, dim=128, rotary=128, pairs="halves",
             scaling="wavelengths"),
        # one long prompt straight into 8 bits, but for its last tokens
        dict(name="write8_1req_64k", op="write8", batch=1, lo=65521, hi=65521, ctx_lo=0, ctx_hi=0,
             hot=1024, q_heads=32, kv_heads=8, dim=128, rotary=128, pairs="halves",
             scaling="none"),
        # one token of a full serving batch
        dict(name="conv_256req_token", op="conv", batch=256, lo=1, hi=1, channels=4352, width=4,
             beside=4160, token=True),
        # a batch of short ragged prompts, half of them continuing a state
        dict(name="conv_16req_short", op="conv", batch=16, lo=1, hi=517, channels=4352, width=4,
             beside=4160, token=False),
        # one long prompt of a wide layer
        dict(name="conv_1req_32k", op="conv", batch=1, lo=32751, hi=32751, channels=6144, width=4,
             beside=4160, token=False),
        # one token of two requests: latency
        dict(name="scan_2req_token", op="scan", batch=2, lo=1, hi=1, heads=4, groups=2, dim=64,
             state=64, f32=True, token=True),
        # one token of a full serving batch
        dict(name="scan_256req_token", op="scan", batch=256, lo=1, hi=1, heads=64, groups=1, dim=64,
             state=128, f32=False, token=True),
        # a batch of short ragged prompts, half of them continuing a state
        dict(name="scan_16req_short", op="scan", batch=16, lo=1, hi=517, heads=64, groups=1, dim=64,
             state=128, f32=False, token=False),
        # one long prompt of a wide layer
        dict(name="scan_1req_32k", op="scan", batch=1, lo=32751, hi=32751, heads=64, groups=8,
             dim=64, state=128, f32=False, token=False),
    ]


def _log(rng, lo, hi):
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_lengths(rng, most):
    """Requests and the range of their new tokens: single tokens, one prompt or a ragged batch."""
    kind = rng.choice(["token", "one", "batch"])
    if kind == "token":
        return True, dict(batch=_log(rng, 1, 256), lo=1, hi=1)
    if kind == "one":
        n = _log(rng, 1, most)
        return False, dict(batch=1, lo=n, hi=n)
    return False, dict(batch=_log(rng, 2, 16), lo=_log(rng, 1, 16), hi=_log(rng, 17, most // 16))


def draw(rng):
    op = rng.choice(["write", "write", "write8", "conv", "conv", "scan", "scan", "scan"])
    token, case = _draw_lengths(rng, 32751)
    if op in ("write", "write8"):
        dim, kvh = rng.choice([64, 128]), _log(rng, 1, 8)
        ctx = 0 if not token and rng.random() < 0.3 else _log(rng, 1, 1000)
        case.update(op=op, ctx_lo=ctx, ctx_hi=ctx and _log(rng, ctx, 4000), kv_heads=kvh,
                    q_heads=kvh * rng.choice([1, 2, 4]), dim=dim, rotary=rng.choice([16, dim // 2, dim, dim]),
                    pairs=rng.choice(["halves", "neighbours"]),
                    scaling=rng.choice(["none", "linear", "parts", "wavelengths"]))
        if op == "write8":
            case["hot"] = rng.choice([0, 1, 64, _log(rng, 1, 1024)])
        return case
    if op == "conv":
        case.update(op=op, channels=8 * _log(rng, 8, 768), width=rng.choice([2, 3, 4, 4]),
                    beside=8 * rng.randint(0, 500), token=token)
        return case
    groups = rng.choice([1, 1, 2, 4, 8])
    case.update(op=op, heads=groups * _log(rng, 1, 64 // groups), groups=groups,
                dim=rng.choice([64, 64, 128]), state=rng.choice([64, 128, 128]),
                f32=token and rng.random() < 0.5, token=token)
    if case["dim"] == 128 and case["heads"] > 32:
        case["heads"] = groups * (32 // groups)
    return case


# A case's lengths follow from the case alone, so that its work does too: spread evenly over the
# logarithm of [lo, hi], in a mixed order.
def _spread(lo, hi, n, order):
    if hi == 0:
        return np.zeros(n, np.int64)
    x = np.exp(np.linspace(math.log(lo), math.log(hi), n)) if n > 1 else np.array([hi])
    return np.clip(np.round(x), lo, hi).astype(np.int64)[np.random.RandomState(order).permutation(n)]


def _new(c):
    return _spread(c["lo"], c["hi"], c["batch"], 17)


def _context(c):
    return _spread(c["ctx_lo"], c["ctx_hi"], c["batch"], 29)


def _warm(c, n):
    """Tokens of a cache of n that are held in 8 bits: whole blocks, the last `hot` tokens not."""
    return np.maximum(n - c["hot"], 0) // BLOCK * BLOCK


def _pages(n):
    return (n + PAGE - 1) // PAGE


# --------------------------------------------------------------- preparing --
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device=DEV, dtype=dtype)


def _int(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _table(rs, need, spare, margin):
    """Pages of each request drawn without replacement, entries behind its last one -1."""
    total = int(need.sum()) + spare
    ids, table, at = rs.permutation(total), np.full((len(need), int(need.max()) + margin), -1), 0
    for r, n in enumerate(need):
        table[r, :n] = ids[at:at + n]
        at += int(n)
    return table, total


def _frequencies(c):
    """Angle that each pair of a rotated head turns by per position, and the factor on both parts."""
    half = c["rotary"] // 2
    i = np.arange(half)
    freq = 10000.0 ** (-i / half)
    factor, trained = 8.0, 4096
    if c["scaling"] == "linear":
        return freq / factor, 1.0
    if c["scaling"] == "parts":
        # pairs of over 32 rotations in the trained length stay, those under one are stretched
        at = half * np.log(trained / (2 * np.pi * np.array([32.0, 1.0]))) / math.log(10000.0)
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), half - 1)
        ramp = np.clip((i - low) / max(high - low, 0.001), 0, 1)
        return freq * (1 - ramp) + freq / factor * ramp, 0.1 * math.log(factor) + 1
    if c["scaling"] == "wavelengths":
        # pairs of over 4 rotations stay, those under one are stretched
        keep = np.clip((trained * freq / (2 * np.pi) - 1) / (4 - 1), 0, 1)
        return freq * keep + freq / factor * (1 - keep), 1.0
    return freq, 1.0


def prepare(case, seed):
    rs, g = np.random.RandomState(seed % (1 << 31)), _gen(seed)
    return dict(write=_prepare_write, write8=_prepare_write, conv=_prepare_conv,
                scan=_prepare_scan)[case["op"]](case, rs, g)


def _prepare_write(c, rs, g):
    new, ctx, hq, hk, d = _new(c), _context(c), c["q_heads"], c["kv_heads"], c["dim"]
    lens, t = new + ctx, int(new.sum())
    table, total = _table(rs, _pages(lens), 5, 1)
    freq, factor = _frequencies(c)
    # the share of a turn that one position adds, as a 64-bit fraction
    turns = np.array([round(f / (2 * math.pi) * 2.0 ** 64) for f in freq.tolist()], dtype=np.uint64)
    rows = _randn(g, t, (hq + 2 * hk) * d)  # one projection's output: queries, keys, values
    s = dict(case=c, q=rows[:, :hq * d].view(t, hq, d), k=rows[:, hq * d:(hq + hk) * d].view(t, hk, d),
             v=rows[:, (hq + hk) * d:].view(t, hk, d), pool_k=_randn(g, total, hk, PAGE, d),
             pool_v=_randn(g, total, hk, PAGE, d), table=_int(table), lens=_int(lens),
             cu=None if c["hi"] == 1 else _int(np.concatenate([[0], np.cumsum(new)])),
             freq=torch.from_numpy(freq).to(DEV), factor=factor,
             turns=torch.from_numpy(turns.view(np.int64)).to(DEV))
    if c["op"] == "write":
        return s
    before, after = _warm(c, ctx), _warm(c, lens)
    qtable, qtotal = _table(rs, after // BLOCK, 5, 1)
    s.update(qtable=_int(qtable), before=_int(before), after=_int(after),
             max_blocks=int((after - before).max()) // BLOCK,
             # earlier blocks: codes and a scale for each block and head
             k8=torch.randint(1, 256, (qtotal, hk, BLOCK, d), generator=g, device=DEV,
                              dtype=torch.uint8),
             v8=torch.randint(1, 256, (qtotal, hk, 2, d, BLOCK // 2), generator=g, device=DEV,
                              dtype=torch.uint8),
             k_scale=torch.rand(qtotal, hk, generator=g, device=DEV) * 0.01 + 0.02,
             v_scale=torch.rand(qtotal, hk, generator=g, device=DEV) * 0.01 + 0.02,
             starts=_int(ctx), max_new=int(new.max()), total=t,
             read_cu=_int(np.concatenate([[0], np.cumsum(new)])))
    return s


def _prepare_conv(c, rs, g):
    new = _new(c)
    t, ch, b = int(new.sum()), c["channels"], c["batch"]
    rows = _randn(g, t, ch + c["beside"])  # a projection's output, of which the layer convolves a part
    return dict(case=c, x=rows[:, c["beside"]:], state=_randn(g, b + 3, c["width"] - 1, ch),
                ids=_int(rs.permutation(b + 3)[:b]), resume=_int(np.arange(b) % 2),
                cu=_int(np.concatenate([[0], np.cumsum(new)])), max_new=int(new.max()),
                weight=torch.randn(ch, c["width"], generator=g, device=DEV) * c["width"] ** -0.5,
                bias=torch.randn(ch, generator=g, device=DEV) * 0.1)


def _prepare_scan(c, rs, g):
    new = _new(c)
    t, b, h, gr, p, n = int(new.sum()), c["batch"], c["heads"], c["groups"], c["dim"], c["state"]
    rows = torch.nn.functional.silu(_randn(g, t, h * p + 2 * gr * n))  # a convolution's output
    # steps from a thousandth to a tenth, each moved by its token; rates from 1 to 16
    step = torch.exp(torch.rand(h, generator=g, device=DEV) * math.log(100) + math.log(1e-3))
    return dict(case=c, x=rows[:, :h * p].view(t, h, p), b=rows[:, h * p:h * p + gr * n].view(t, gr, n),
                c=rows[:, h * p + gr * n:].view(t, gr, n), dt=_randn(g, t, h) * 0.7,
                state=_randn(g, b + 3, h, p, n, dtype=torch.float32) * 0.1,
                ids=_int(rs.permutation(b + 3)[:b]), resume=_int(np.arange(b) % 2),
                cu=_int(np.concatenate([[0], np.cumsum(new)])), max_new=int(new.max()),
                rate=-1 - 15 * torch.rand(h, generator=g, device=DEV),
                skip=1 + 0.2 * torch.randn(h, generator=g, device=DEV),
                dt_bias=step + torch.log(-torch.expm1(-step)),
                dtype=torch.float32 if c["f32"] else torch.bfloat16)


# ----------------------------------------------------------------- running --
def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _places(s):
    """(request, position) of each new token."""
    cu = s.get("read_cu", s["cu"])
    new = torch.ones_like(s["lens"]) if cu is None else cu[1:] - cu[:-1]
    req = torch.repeat_interleave(torch.arange(len(new), device=DEV), new,
                                  output_size=s["k"].shape[0])
    first = torch.cumsum(new, 0) - s["lens"]  # row of a token less its position
    return req, torch.arange(len(req), device=DEV) - first[req]


def _rotated(s, x, pos):
    c = s["case"]
    r = c["rotary"]
    angle = pos.double()[:, None] * s["freq"]  # of far positions: in 64 bits
    cos = (torch.cos(angle) * s["factor"]).float()[:, None]
    sin = (torch.sin(angle) * s["factor"]).float()[:, None]
    y = x.float()
    if c["pairs"] == "halves":
        a, b = y[..., :r // 2], y[..., r // 2:r]
        parts = [a * cos - b * sin, b * cos + a * sin, y[..., r:]]
        return torch.cat(parts, -1).bfloat16()
    a, b = y[..., 0:r:2], y[..., 1:r:2]
    turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, y[..., r:]], -1).bfloat16()


def _plain_write(s):
    req, pos = _places(s)
    page = s["table"][req, pos // PAGE].long()
    s["pool_k"][page, :, pos % PAGE] = _rotated(s, s["k"], pos)
    s["pool_v"][page, :, pos % PAGE] = s["v"]
    return dict(q=_rotated(s, s["q"], pos), k=s["pool_k"], v=s["pool_v"])


def _rope(phs, s):
    return phs.Rope(s["turns"], interleaved=s["case"]["pairs"] == "neighbours", factor=s["factor"])


def _own_write(s):
    import paged_hybrid_sliding_gb300 as phs
    q = phs.kv_write_paged(phs.PagedPool(s["pool_k"], s["pool_v"]), s["k"], s["v"], s["table"],
                           s["lens"], cu_seqlens=s["cu"], q=s["q"], rope=_rope(phs, s))
    return dict(q=q, k=s["pool_k"], v=s["pool_v"])


# Token at byte p of a half block's stored row of values: pairs of tokens 8 apart side by side.
_VT = [2 * (p >> 2) + (p & 1) + 8 * ((p >> 1) & 1) for p in range(16)]


def _plain_write8(s):
    c = s["case"]
    hk, d, b = c["kv_heads"], c["dim"], c["batch"]
    table, qtable = s["table"].long(), s["qtable"].long()
    req, pos = _places(s)
    # every new token into its page, then the whole blocks that got old out of the pages
    page = table[req, pos // PAGE]
    k_new = _rotated(s, s["k"], pos)
    warm = pos < s["after"][req]
    keep_k, keep_v = s["pool_k"][page, :, pos % PAGE], s["pool_v"][page, :, pos % PAGE]
    s["pool_k"][page, :, pos % PAGE] = k_new
    s["pool_v"][page, :, pos % PAGE] = s["v"]
    first, count = s["before"].long() // BLOCK, (s["after"] - s["before"]).long() // BLOCK
    row = torch.repeat_interleave(torch.arange(b, device=DEV), count)
    block = torch.arange(len(row), device=DEV) - (torch.cumsum(count, 0) - count)[row] + first[row]
    to = qtable[row, block]
    pages = table[row[:, None], 2 * block[:, None] + torch.arange(2, device=DEV)]
    order = torch.tensor(_VT, device=DEV)
    for pool, codes, scales in (("pool_k", "k8", "k_scale"), ("pool_v", "v8", "v_scale")):
        x = s[pool][pages].float().transpose(1, 2).reshape(-1, hk, BLOCK, d)
        scale = x.abs().amax((2, 3)) / 127
        y = torch.round(x / scale.clamp(min=1e-37)[..., None, None])  # (zeros have a scale of zero)
        y = (y.clamp(-127, 127) + 128).to(torch.uint8)
        if codes == "v8":
            y = y.view(-1, hk, 2, PAGE, d)[:, :, :, order].transpose(-1, -2)
        s[codes][to] = y
        s[scales][to] = scale
    # pages keep what they held where a token went straight into 8 bits
    s["pool_k"][page, :, pos % PAGE] = torch.where(warm[:, None, None], keep_k, k_new)
    s["pool_v"][page, :, pos % PAGE] = torch.where(warm[:, None, None], keep_v, s["v"])
    # the new tokens as the cache now holds them
    qpage = torch.where(warm, qtable[req, torch.where(warm, pos // BLOCK, 0)], 0)
    at, half = pos % BLOCK, pos % BLOCK // PAGE
    inverse = torch.empty_like(order)
    inverse[order] = torch.arange(PAGE, device=DEV)
    k8 = (s["k8"][qpage, :, at].float() - 128) * s["k_scale"][qpage][..., None]
    v8 = s["v8"][qpage, :, half, :, inverse[pos % PAGE]].float() - 128
    v8 = v8 * s["v_scale"][qpage][..., None]
    k = torch.where(warm[:, None, None], k8, s["pool_k"][page, :, pos % PAGE].float())
    v = torch.where(warm[:, None, None], v8, s["pool_v"][page, :, pos % PAGE].float())
    return dict(q=_rotated(s, s["q"], pos), k=k.bfloat16(), v=v.bfloat16(), pool_k=s["pool_k"],
                pool_v=s["pool_v"], k_scale=s["k_scale"], v_scale=s["v_scale"])


def _own_write8(s):
    import paged_hybrid_sliding_gb300 as phs
    pool = phs.PagedPool(s["pool_k"], s["pool_v"])
    int8 = phs.Int8Pool(s["k8"], s["v8"], s["k_scale"], s["v_scale"])
    q = phs.kv_write_paged(pool, s["k"], s["v"], s["table"], s["lens"], cu_seqlens=s["cu"], q=s["q"],
                           rope=_rope(phs, s), int8=int8, qtable=s["qtable"],
                           qlens_before=s["before"], qlens=s["after"], max_qblocks=s["max_blocks"])
    k, v = phs.kv_read_paged(pool, s["table"], s["starts"], s["read_cu"], s["total"], s["max_new"],
                             int8=int8, qtable=s["qtable"], qlens=s["after"])
    return dict(q=q, k=k, v=v, pool_k=s["pool_k"], pool_v=s["pool_v"], k_scale=s["k_scale"],
                v_scale=s["v_scale"])


def _padded(s, x, n):
    """Packed rows as [batch, n, ...], zeros behind each request's last; and which rows are real."""
    cu = s["cu"].long()
    t = torch.arange(n, device=DEV)
    real = t < (cu[1:] - cu[:-1])[:, None]
    rows = x[torch.where(real, cu[:-1, None] + t, 0)]
    return torch.where(real.view(*real.shape, *[1] * (x.dim() - 1)), rows, 0), real


def _plain_conv(s):
    c = s["case"]
    w, ids = c["width"], s["ids"].long()
    x, real = _padded(s, s["x"], s["max_new"])
    first = s["state"][ids]
    if not c["token"]:
        first = torch.where(s["resume"][:, None, None] != 0, first, 0)
    x = torch.cat([first, x], 1)  # token t at row w - 1 + t
    y = s["bias"] + sum(x[:, k:k + s["max_new"]].float() * s["weight"][:, k] for k in range(w))
    y = (y * torch.sigmoid(y))[real].bfloat16()
    last = (s["cu"][1:] - s["cu"][:-1]).long()[:, None] + torch.arange(w - 1, device=DEV)
    s["state"][ids] = x.gather(1, last[..., None].expand(-1, -1, x.shape[2]))
    return dict(out=y, state=s["state"])


def _own_conv(s):
    import paged_hybrid_sliding_gb300 as phs
    pool, weights = phs.ConvPool(s["state"]), phs.ConvWeights(s["weight"], s["bias"], silu=True)
    if s["case"]["token"]:
        out = phs.causal_conv_decode(s["x"], pool, weights, state_ids=s["ids"])
    else:
        out = phs.causal_conv_prompt(s["x"], s["cu"], pool, weights, state_ids=s["ids"],
                                     resume=s["resume"])
    return dict(out=out, state=s["state"])


def _softplus(x):
    return x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))


def _plain_scan(s):
    c = s["case"]
    h, gr, p, n = c["heads"], c["groups"], c["dim"], c["state"]
    nb, ids, size = c["batch"], s["ids"].long(), 64
    first = s["state"][ids]
    dt = _softplus(s["dt"].double() + s["dt_bias"])
    if c["token"]:
        b = s["b"].float().repeat_interleave(h // gr, 1)
        cc = s["c"].float().repeat_interleave(h // gr, 1)
        x = s["x"].float()
        state = torch.exp(dt * s["rate"]).float()[..., None, None] * first
        state = state + (dt.float()[..., None] * x)[..., None] * b[:, :, None]
        y = torch.einsum("bhpn,bhn->bhp", state, cc) + s["skip"][:, None] * x
        s["state"][ids] = state
        return dict(out=y.to(s["dtype"]), state=s["state"])
    first = torch.where(s["resume"][:, None, None, None] != 0, first, 0.0)
    nc = -(-s["max_new"] // size)  # chunks
    x, real = _padded(s, s["x"], nc * size)
    x = x.float().view(nb, nc, size, h, p)
    b = _padded(s, s["b"], nc * size)[0].float().view(nb, nc, size, gr, n)
    cc = _padded(s, s["c"], nc * size)[0].float().view(nb, nc, size, gr, n)
    dt = _padded(s, dt, nc * size)[0].view(nb, nc, size, h)  # padding decays nothing
    log = torch.cumsum(dt * s["rate"], 2)  # decay from a chunk's start through each token: 64 bits
    i = torch.arange(size, device=DEV)
    w = (log[:, :, :, None] - log[:, :, None]).masked_fill((i[:, None] < i)[..., None], -math.inf)
    w = torch.exp(w).float() * dt.float()[:, :, None]
    g = torch.einsum("bcign,bcjgn->bcijg", cc, b)
    w = (w.view(nb, nc, size, size, gr, -1) * g[..., None]).view(nb, nc, size, size, h)
    y = torch.einsum("bcijh,bcjhp->bcihp", w, x)
    del w, g
    # the chunks' own states, summed with their decay into the state before each chunk
    end = log[:, :, -1]
    left = (torch.exp(end[:, :, None] - log) * dt).float()
    add = torch.einsum("bcjghp,bcjgn->bcghpn", (left[..., None] * x).view(nb, nc, size, gr, -1, p), b)
    total = torch.cumsum(end, 1)
    ch = torch.arange(nc, device=DEV)
    d = (total - end)[:, :, None] - total[:, None]
    d = torch.exp(d.masked_fill((ch[:, None] <= ch)[..., None], -math.inf)).float()
    before = torch.einsum("bcmh,bmhpn->bchpn", d, add.view(nb, nc, h, p, n))
    before = before + torch.exp(total - end).float()[..., None, None] * first[:, None]
    more = torch.einsum("bcign,bcghpn->bcighp", cc, before.view(nb, nc, gr, -1, p, n))
    y = y + torch.exp(log).float()[..., None] * more.reshape(nb, nc, size, h, p)
    y = y + s["skip"][:, None] * x
    last = torch.exp(end[:, -1]).float()[..., None, None]
    s["state"][ids] = last * before[:, -1] + add[:, -1].reshape(nb, h, p, n)
    return dict(out=y.reshape(nb, -1, h, p)[real].bfloat16(), state=s["state"])


def _own_scan(s):
    import paged_hybrid_sliding_gb300 as phs
    pool = phs.ScanPool(s["state"])
    weights = phs.ScanWeights(s["rate"], skip=s["skip"], dt_bias=s["dt_bias"])
    if s["case"]["token"]:
        out = phs.selective_scan_decode(s["x"], s["dt"], s["b"], s["c"], pool, weights,
                                        state_ids=s["ids"], out_dtype=s["dtype"])
    else:
        out = phs.selective_scan_prompt(s["x"], s["dt"], s["b"], s["c"], s["cu"], s["max_new"], pool,
                                        weights, state_ids=s["ids"], resume=s["resume"])
    return dict(out=out, state=s["state"])


_plain = dict(write=_plain_write, write8=_plain_write8, conv=_plain_conv, scan=_plain_scan)
_own = dict(write=_own_write, write8=_own_write8, conv=_own_conv, scan=_own_scan)


# -------------------------------------------------------------------- work --
def work(c):
    new = _new(c)
    t, b = int(new.sum()), c["batch"]
    if c["op"] in ("write", "write8"):
        d, hq, hk = c["dim"], c["q_heads"], c["kv_heads"]
        size, turned = 4 * t * (hq + 2 * hk) * d, 3 * t * (hq + hk) * c["rotary"]
        if c["op"] == "write":
            return dict(bytes=size, flops=turned)
        # tokens that got old: read from the pages or the new rows, written and read again in 8 bits
        lens, ctx = _context(c) + new, _context(c)
        before, after = _warm(c, ctx), _warm(c, lens)
        moved = int((after - before).sum())
        fresh = int(np.maximum(after - np.maximum(ctx, before), 0).sum())  # new and old at once
        cell = 2 * hk * d
        size = 4 * t * hq * d + cell * (2 * t + 2 * (moved - fresh) + moved + 2 * (t - fresh))
        size += cell * (fresh + 2 * (t - fresh) + 2 * t)  # reading back
        return dict(bytes=size, flops=turned + 4 * moved * cell)
    if c["op"] == "conv":
        ch, w = c["channels"], c["width"]
        return dict(bytes=4 * ch * (t + b * (w - 1) + w + 1), flops=t * ch * (2 * w + 4))
    h, gr, p, n = c["heads"], c["groups"], c["dim"], c["state"]
    io = t * (h * p * (6 if c["f32"] else 4) + 4 * gr * n + 2 * h)
    # a prompt reads the state where it continues one
    state = b * h * p * n * (8 if c["token"] else 6)
    return dict(bytes=io + state, flops=4 * t * h * p * n)


# ------------------------------------------------- the definitions, 64 bits --
def exact(case, seed):
    s = prepare(case, seed)
    return dict(write=_exact_write, write8=_exact_write8, conv=_exact_conv,
                scan=_exact_scan)[case["op"]](s)


def _exact_turn(s, x, pos):
    """One request's rows, rotated pair by pair as complex numbers."""
    r = s["case"]["rotary"]
    turn = torch.polar(torch.full_like(s["freq"], s["factor"]).expand(len(pos), -1),
                       pos.double()[:, None] * s["freq"])[:, None]
    y = x.double().clone()
    lo, hi = (slice(0, r // 2), slice(r // 2, r)) if s["case"]["pairs"] == "halves" else \
        (slice(0, r, 2), slice(1, r, 2))
    z = torch.complex(y[..., lo], y[..., hi]) * turn
    y[..., lo], y[..., hi] = z.real, z.imag
    return y


def _exact_rows(s):
    """For each request: its row of the tables, its new tokens' rows and positions."""
    at = 0
    for r, (n, m) in enumerate(zip(s["lens"].tolist(), _new(s["case"]).tolist())):
        yield r, slice(at, at + m), torch.arange(n - m, n, device=DEV)
        at += m


def _exact_write(s):
    k, v = s["pool_k"].double(), s["pool_v"].double()
    q = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    for r, rows, pos in _exact_rows(s):
        page = s["table"][r].long()[pos // PAGE]
        k[page, :, pos % PAGE] = _exact_turn(s, s["k"][rows], pos)
        v[page, :, pos % PAGE] = s["v"][rows].double()
        q[rows] = _exact_turn(s, s["q"][rows], pos)
    return dict(q=q, k=k, v=v)


def _exact_write8(s):
    pool = dict(k=s["pool_k"].double(), v=s["pool_v"].double())
    scale = dict(k=s["k_scale"].double(), v=s["v_scale"].double())
    got = {x: torch.empty(s["k"].shape, dtype=torch.float64, device=DEV) for x in "kv"}
    q = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    for r, rows, pos in _exact_rows(s):
        q[rows] = _exact_turn(s, s["q"][rows], pos)
        n, new, lo, hi = int(s["lens"][r]), int(pos[0]), int(s["before"][r]), int(s["after"][r])
        tokens = torch.arange(n, device=DEV)
        page = s["table"][r].long()[tokens // PAGE]
        for x, fresh in (("k", _exact_turn(s, s["k"][rows], pos)), ("v", s["v"][rows].double())):
            seq = pool[x][page, :, tokens % PAGE]  # [tokens, heads, dim]
            seq[new:] = fresh.bfloat16().double()  # the cache holds bf16, and codes of that
            cold = max(hi, new)
            pool[x][page[cold:], :, tokens[cold:] % PAGE] = fresh[cold - new:]
            blocks = seq[lo:hi].view(-1, BLOCK, *seq.shape[1:])
            a = blocks.abs().amax((1, 3)) / 127
            codes = torch.round(blocks / a[:, None, :, None])
            scale[x][s["qtable"][r, lo // BLOCK:hi // BLOCK].long()] = a
            held = torch.cat([seq[:lo], (codes * a[:, None, :, None]).flatten(0, 1), seq[hi:]])
            got[x][rows] = held[new:]
    return dict(q=q, k=got["k"], v=got["v"], pool_k=pool["k"], pool_v=pool["v"], k_scale=scale["k"],
                v_scale=scale["v"])


def _exact_conv(s):
    w, state = s["case"]["width"], s["state"].double()
    out = torch.empty(s["x"].shape, dtype=torch.float64, device=DEV)
    cu = s["cu"].tolist()
    for r, i in enumerate(s["ids"].tolist()):
        first = state[i] if s["case"]["token"] or int(s["resume"][r]) else torch.zeros_like(state[i])
        x = torch.cat([first, s["x"][cu[r]:cu[r + 1]].double()])
        y = (x.unfold(0, w, 1) * s["weight"].double()).sum(-1) + s["bias"].double()
        out[cu[r]:cu[r + 1]] = y / (1 + torch.exp(-y))
        state[i] = x[len(x) - (w - 1):]
    return dict(out=out, state=state)


def _exact_scan(s):
    c = s["case"]
    h, gr, p, n = c["heads"], c["groups"], c["dim"], c["state"]
    # a step is about ten launches, and 12 passes over the states at 3 TB/s in 64 bits
    if s["max_new"] * (7e-5 + c["batch"] * h * p * n * 8 * 12 / 3e12) > 15:
        return None
    cu, ids = s["cu"].long(), s["ids"].long()
    rate, skip, bias = (s[x].double() for x in ("rate", "skip", "dt_bias"))
    state = s["state"].double()
    now = state[ids] if c["token"] else state[ids] * (s["resume"] != 0)[:, None, None, None]
    order = torch.argsort(cu[1:] - cu[:-1], descending=True)
    lens = (cu[1:] - cu[:-1])[order].tolist()
    now, start = now[order], cu[:-1][order]
    out = torch.empty(s["x"].shape, dtype=torch.float64, device=DEV)
    live = len(lens)
    for t in range(s["max_new"]):
        while lens[live - 1] <= t:
            live -= 1
        at = start[:live] + t
        dt = torch.log(1 + torch.exp(s["dt"][at].double() + bias))
        x = s["x"][at].double()
        b = s["b"][at].double()[:, :, None].expand(-1, -1, h // gr, -1).reshape(live, h, 1, n)
        cc = s["c"][at].double()[:, :, None].expand(-1, -1, h // gr, -1).reshape(live, h, n, 1)
        now[:live] *= torch.exp(dt * rate)[..., None, None]
        now[:live] += (dt[..., None] * x)[..., None] * b
        out[at] = (now[:live] @ cc)[..., 0] + skip[:, None] * x
    state[ids[order]] = now
    return dict(out=out, state=state)
