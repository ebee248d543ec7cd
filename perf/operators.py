"""Measured cases of the cache and layer operators of a hybrid serving stack:

  fork       free the rows of dropped continuations of a paged cache, then fork
             surviving requests into them (whole pages shared, the last partial
             page copied, in every layer's pool)
  compact    move the live pages of a fragmented pool to its lowest page ids and
             rewrite block tables and reference counts
  diff       differential attention of one new token over the paged cache
  recur      linear attention with a decay per head, one new token per request
  prompt     the same over whole prompts (ragged, packed), states carried along

`run` computes them in plain torch where `own` is false and through the
package's entry points where it is true.
"""
import math

import numpy as np
import torch

own = False

PAGE = 16
DEV = "cuda"


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # a beam-search step of two short conversations on a two-layer stack: latency
        dict(name="fork_4to4_2layers", op="fork", parents=4, children=4, lo=37, hi=2000, layers=2,
             heads=2, dim=64, spare=64),
        # 64 requests, three continuations sampled from each, ten Full layers
        dict(name="fork_64to192_10layers", op="fork", parents=64, children=192, lo=1024, hi=16384,
             layers=10, heads=8, dim=128, spare=500),
        # defragmenting a small pool between two steps
        dict(name="compact_512pages_2layers", op="compact", rows=12, lo=1, hi=700, layers=2,
             heads=2, dim=64, pages=512, moves=61, shared=3),
        # giving back the upper part of a large pool after many requests ended
        dict(name="compact_16384pages_10layers", op="compact", rows=48, lo=1024, hi=8191, layers=10,
             heads=8, dim=128, pages=16384, moves=3001, shared=16),
        # one decode step of two short requests with the append: latency
        dict(name="diff_2req_short_f32", op="diff", batch=2, lo=37, hi=201, heads=4, value_heads=2,
             dim=64, append=True, f32=True, norm=True),
        # a mixed batch of short and ordinary conversations, append fused
        dict(name="diff_16req_4k", op="diff", batch=16, lo=1, hi=4097, heads=16, value_heads=4,
             dim=128, append=True, f32=False, norm=True),
        # a full serving batch, lengths 1K to 32K
        dict(name="diff_64req_32k", op="diff", batch=64, lo=1024, hi=32768, heads=16, value_heads=4,
             dim=128, append=True, f32=False, norm=True),
        # one long document
        dict(name="diff_1req_250k", op="diff", batch=1, lo=250001, hi=250001, heads=32,
             value_heads=4, dim=64, append=False, f32=False, norm=False),
        # one token of two requests: latency
        dict(name="recur_2req", op="recur", batch=2, q_heads=4, kv_heads=2, dim=64, f32=True),
        # one token of a full serving batch
        dict(name="recur_256req", op="recur", batch=256, q_heads=32, kv_heads=32, dim=128, f32=False),
        # a batch of short ragged prompts, half of them continuing a state
        dict(name="prompt_16req_short", op="prompt", batch=16, lo=1, hi=517, q_heads=32, kv_heads=8,
             dim=128),
        # one long prompt
        dict(name="prompt_1req_32k", op="prompt", batch=1, lo=32751, hi=32751, q_heads=32,
             kv_heads=32, dim=128),
    ]


def _log(rng, lo, hi):
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["fork", "compact", "diff", "diff", "recur", "prompt", "prompt"])
    dim = rng.choice([64, 128])
    if op == "fork":
        parents = _log(rng, 1, 64)
        return dict(op=op, parents=parents, children=_log(rng, 1, 3 * parents), lo=_log(rng, 1, 900),
                    hi=_log(rng, 1000, 16384), layers=_log(rng, 1, 10), heads=_log(rng, 1, 8),
                    dim=dim, spare=_log(rng, 64, 500))
    if op == "compact":
        rows, hi = _log(rng, 1, 48), _log(rng, 40, 8191)
        case = dict(op=op, rows=rows, lo=_log(rng, 1, 40), hi=hi, layers=_log(rng, 1, 10),
                    heads=_log(rng, 1, 8), dim=dim, pages=0, moves=0, shared=rng.choice([0, 1, 2]))
        live = _live_pages(case)
        case["pages"] = live + _log(rng, 1, 8000)
        case["moves"] = rng.randint(0, min(live, case["pages"] - live, 3000))
        return case
    if op == "diff":
        vh = _log(rng, 1, 4)
        return dict(op=op, batch=_log(rng, 1, 64), lo=_log(rng, 1, 1000), hi=_log(rng, 1024, 32768),
                    heads=vh * rng.choice([1, 2, 3, 4, 8, 16]), value_heads=vh, dim=dim,
                    append=rng.random() < 0.5, f32=rng.random() < 0.5, norm=rng.random() < 0.7)
    kvh = _log(rng, 1, 32)
    qh = kvh * rng.choice([1, 1, 2, 4] if kvh <= 8 else [1])
    if op == "recur":
        return dict(op=op, batch=_log(rng, 1, 256), q_heads=qh, kv_heads=kvh, dim=dim,
                    f32=rng.random() < 0.5)
    if rng.random() < 0.5:
        n = _log(rng, 1, 32751)
        return dict(op=op, batch=1, lo=n, hi=n, q_heads=qh, kv_heads=kvh, dim=dim)
    return dict(op=op, batch=_log(rng, 2, 16), lo=_log(rng, 1, 16), hi=_log(rng, 17, 2000),
                q_heads=qh, kv_heads=kvh, dim=dim)


# A case's lengths follow from the case alone, so that its work does too: spread evenly over the
# logarithm of [lo, hi], in a mixed order.
def _lens(case, n):
    lo, hi = case["lo"], case["hi"]
    x = np.exp(np.linspace(math.log(lo), math.log(hi), n)) if n > 1 else np.array([hi])
    x = np.clip(np.round(x), lo, hi).astype(np.int64)
    return x[np.random.RandomState(17).permutation(n)]


def _pages(n):
    return (n + PAGE - 1) // PAGE


def _live_pages(case):
    own_pages = np.maximum(_pages(_lens(case, case["rows"])) - case["shared"], 0)
    return int(own_pages.sum()) + int(min(case["shared"], _pages(_lens(case, case["rows"])).max()))


# --------------------------------------------------------------- preparing --
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device=DEV, dtype=dtype)


def _int(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _pool(g, pages, heads, dim):
    return _randn(g, pages, heads, PAGE, dim), _randn(g, pages, heads, PAGE, dim)


def prepare(case, seed):
    rs, g = np.random.RandomState(seed % (1 << 31)), _gen(seed)
    return dict(fork=_prepare_fork, compact=_prepare_compact, diff=_prepare_diff,
                recur=_prepare_recur, prompt=_prepare_prompt)[case["op"]](case, rs, g)


def _prepare_fork(c, rs, g):
    np_, nc = c["parents"], c["children"]
    lens = np.concatenate([_lens(c, np_), _lens(c, nc)[rs.permutation(nc)]])
    need = _pages(lens)
    total = int(need.sum()) + c["spare"]
    ids = rs.permutation(total)
    width = int(need.max())
    table = np.full((np_ + nc, width), -1)
    at = 0
    for r in range(np_ + nc):
        table[r, :need[r]] = ids[at:at + need[r]]
        at += int(need[r])
    counts = np.zeros(total, np.int64)
    counts[ids[:at]] = 1
    s = dict(case=c, pools=[_pool(g, total, c["heads"], c["dim"]) for _ in range(c["layers"])],
             table=_int(table), lens=_int(lens), counts=_int(counts),
             src=_int(np.arange(nc) % np_), dst=_int(np_ + rs.permutation(nc)))
    return s


def _prepare_compact(c, rs, g):
    lens = _lens(c, c["rows"])
    need, live, total = _pages(lens), _live_pages(c), c["pages"]
    holes = rs.permutation(live)[:c["moves"]]
    upper = live + rs.permutation(total - live)[:c["moves"]]
    ids = rs.permutation(np.concatenate([np.setdiff1d(np.arange(live), holes), upper]))
    shared = min(c["shared"], int(need.max()))
    table = np.full((c["rows"], int(need.max()) + 3), -1)
    counts = np.zeros(total, np.int64)
    at = shared
    for r in range(c["rows"]):  # the first pages of every row are shared
        k = min(shared, int(need[r]))
        table[r, :k] = ids[:k]
        table[r, k:need[r]] = ids[at:at + need[r] - k]
        at += int(need[r]) - k
        counts[table[r, :need[r]]] += 1
    s = dict(case=c, pools=[_pool(g, total, c["heads"], c["dim"]) for _ in range(c["layers"])],
             table=_int(table), lens=_int(lens), counts=_int(counts))
    s.update(table_out=torch.empty_like(s["table"]), counts_out=torch.empty_like(s["counts"]),
             page_map=torch.empty_like(s["counts"]),
             num_live=torch.empty(1, dtype=torch.int32, device=DEV))
    return s


def _prepare_diff(c, rs, g):
    b, h, vh, d = c["batch"], c["heads"], c["value_heads"], c["dim"]
    lens = _lens(c, b)
    need = _pages(lens)
    total = int(need.sum()) + 5
    ids = rs.permutation(total)
    table = np.full((b, int(need.max()) + 1), -1)
    at = 0
    for r in range(b):
        table[r, :need[r]] = ids[at:at + need[r]]
        at += int(need[r])
    k, v = _pool(g, total, 2 * vh, d)
    # logits of standard deviation 1.5: maps that are neither flat nor one-hot
    q = _randn(g, b, 2 * h, d) * 1.5
    s = dict(case=c, k=k, v=v, q=q, table=_int(table), lens=_int(lens), max_len=int(lens.max()),
             lam=[torch.randn(d, generator=g, device=DEV) * 0.1 for _ in range(4)], lam_init=0.55,
             norm=1 + 0.2 * torch.randn(2 * d, generator=g, device=DEV) if c["norm"] else None,
             eps=1e-5, dtype=torch.float32 if c["f32"] else torch.bfloat16,
             k_new=_randn(g, b, 2 * vh, d) if c["append"] else None,
             v_new=_randn(g, b, 2 * vh, d) if c["append"] else None)
    return s


# One decay rate per head, from a memory of about two tokens to one of thousands.
def _decay(heads, g):
    rate = torch.exp(torch.linspace(math.log(0.7), math.log(2e-4), heads, device=DEV)
                     + 0.05 * torch.randn(heads, generator=g, device=DEV))
    return (-rate).float()


def _prepare_recur(c, rs, g):
    b, d = c["batch"], c["dim"]
    slots = b + 3
    s = dict(case=c, state=_randn(g, slots, c["kv_heads"], d, d, dtype=torch.float32),
             ids=_int(rs.permutation(slots)[:b]), decay=_decay(c["kv_heads"], g),
             q=_randn(g, b, c["q_heads"], d), k=_randn(g, b, c["kv_heads"], d) * d ** -0.5,
             v=_randn(g, b, c["kv_heads"], d), scale=d ** -0.5,
             dtype=torch.float32 if c["f32"] else torch.bfloat16)
    return s


def _prepare_prompt(c, rs, g):
    b, d = c["batch"], c["dim"]
    lens = _lens(c, b)
    slots, t = b + 3, int(lens.sum())
    s = dict(case=c, state=_randn(g, slots, c["kv_heads"], d, d, dtype=torch.float32),
             ids=_int(rs.permutation(slots)[:b]), decay=_decay(c["kv_heads"], g),
             resume=_int(np.arange(b) % 2), cu=_int(np.concatenate([[0], np.cumsum(lens)])),
             max_len=int(lens.max()), q=_randn(g, t, c["q_heads"], d),
             k=_randn(g, t, c["kv_heads"], d) * d ** -0.5, v=_randn(g, t, c["kv_heads"], d),
             scale=d ** -0.5)
    return s


# ----------------------------------------------------------------- running --
def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _fork_outputs(s):
    return dict(table=s["table"], lens=s["lens"], counts=s["counts"], pools=s["pools"])


def _compact_outputs(s):
    return dict(table=s["table_out"], counts=s["counts_out"], page_map=s["page_map"],
                num_live=s["num_live"], pools=s["pools"])


def _plain_fork(s):
    table, lens, counts = s["table"], s["lens"], s["counts"]
    src, dst = s["src"].long(), s["dst"].long()
    col = torch.arange(table.shape[1], device=DEV)
    # free the rows that the new continuations take
    held = col < _pages(lens[dst])[:, None]
    counts.index_add_(0, table[dst].clamp(min=0).flatten().long(), -held.flatten().int())
    lens[dst] = 0
    # share whole pages; a fresh page, the lowest free one, for the last partial page
    n = lens[src]
    part = n % PAGE != 0
    last = torch.where(part, n // PAGE, (n // PAGE - 1).clamp(min=0)).long()
    rank = torch.cumsum(part, 0) - 1
    free = torch.sort((counts != 0).int(), stable=True).indices
    rows = table[src]
    old = rows.gather(1, last[:, None])[:, 0].clamp(min=0).long()
    fresh = torch.where(part, free[rank.clamp(min=0)], old)
    whole = col < (n // PAGE)[:, None]
    counts.index_add_(0, rows.clamp(min=0).flatten().long(), whole.flatten().int())
    counts.index_add_(0, fresh, part.int())
    for k, v in s["pools"]:
        k[fresh] = k[old]
        v[fresh] = v[old]
    rows = torch.where(part[:, None] & (col == last[:, None]), fresh[:, None].int(), rows)
    table[dst] = torch.where(col < _pages(n)[:, None], rows, table[dst])
    lens[dst] = n
    return _fork_outputs(s)


def _own_fork(s):
    import paged_hybrid_sliding_gb300 as phs
    phs.pages_free(s["table"], s["lens"], s["counts"], s["dst"])
    phs.pages_fork([phs.PagedPool(k, v) for k, v in s["pools"]], s["table"], s["lens"],
                   s["counts"], s["src"], s["dst"])
    return _fork_outputs(s)


def _plain_compact(s):
    table, counts = s["table"], s["counts"]
    total = counts.shape[0]
    live = counts > 0
    ids = torch.arange(total, device=DEV)
    num = live.sum()
    # the highest live page goes to the lowest hole, and so on
    mover, hole = live & (ids >= num), ~live & (ids < num)
    moves = mover.sum()
    from_ = torch.sort(torch.where(mover, ids, -1), descending=True).values
    to = torch.sort(torch.where(hole, ids, total)).values
    at = ids < moves
    src, dst = torch.where(at, from_, 0), torch.where(at, to, 0)  # past the moves: page 0 to itself
    mapped = torch.where(live, ids, -1)
    mapped = torch.cat([mapped, mapped.new_zeros(1)])
    mapped[torch.where(at, from_, total)] = torch.where(at, to, 0)
    mapped = mapped[:total]
    s["page_map"].copy_(mapped)
    s["num_live"].copy_(num)
    new = torch.cat([torch.where(mover, 0, counts), counts.new_zeros(1)])
    new[torch.where(at, to, total)] = torch.where(at, counts[src], 0)
    s["counts_out"].copy_(new[:total])
    held = torch.arange(table.shape[1], device=DEV) < _pages(s["lens"])[:, None]
    s["table_out"].copy_(torch.where(held, mapped[table.clamp(min=0).long()].int(), table))
    most = s["case"]["moves"]
    src, dst = src[:most], dst[:most]
    for k, v in s["pools"]:
        k[dst] = k[src]
        v[dst] = v[src]
    return _compact_outputs(s)


def _own_compact(s):
    import paged_hybrid_sliding_gb300 as phs
    phs.pages_compact([phs.PagedPool(k, v) for k, v in s["pools"]], s["table"], s["lens"],
                      s["counts"], block_table_out=s["table_out"],
                      page_refcount_out=s["counts_out"], page_map=s["page_map"],
                      num_live=s["num_live"])
    return _compact_outputs(s)


def _lambda(s, dtype):
    a, b, c, d = (x.to(dtype) for x in s["lam"])
    return torch.exp((a * b).sum()) - torch.exp((c * d).sum()) + s["lam_init"]


def _plain_diff(s):
    c = s["case"]
    b, h, vh, d = c["batch"], c["heads"], c["value_heads"], c["dim"]
    lens, table = s["lens"].long(), s["table"].long()
    if c["append"]:
        page = table.gather(1, (lens - 1)[:, None] // PAGE)[:, 0]
        s["k"][page, :, (lens - 1) % PAGE] = s["k_new"]
        s["v"][page, :, (lens - 1) % PAGE] = s["v_new"]
    at = table[:, :_pages(s["max_len"])].clamp(min=0)
    t = at.shape[1] * PAGE
    k = s["k"][at].permute(0, 2, 1, 3, 4).reshape(b, vh, 2, t, d).float()
    q = s["q"].view(b, vh, h // vh, 2, d).float()
    w = torch.einsum("bhgmd,bhmtd->bhgmt", q, k) * d ** -0.5
    del k
    w = w.masked_fill(torch.arange(t, device=DEV) >= lens[:, None, None, None, None], -math.inf)
    w = torch.exp(w - w.amax(-1, keepdim=True))
    w = w / w.sum(-1, keepdim=True)
    w = w[:, :, :, 0] - _lambda(s, torch.float32) * w[:, :, :, 1]
    v = s["v"][at].permute(0, 2, 1, 3, 4).reshape(b, vh, 2, t, d).float()
    o = torch.einsum("bhgt,bhmtd->bhgmd", w, v).reshape(b, h, 2 * d)
    if s["norm"] is not None:
        o = o * torch.rsqrt(o.square().mean(-1, keepdim=True) + s["eps"]) * s["norm"]
        o = o * (1 - s["lam_init"])
    return dict(out=o.to(s["dtype"]), k=s["k"], v=s["v"])


def _own_diff(s):
    import paged_hybrid_sliding_gb300 as phs
    weights = phs.DiffWeights(*s["lam"], lambda_init=s["lam_init"], norm_weight=s["norm"],
                              norm_eps=s["eps"])
    out = phs.attn_decode_diff_paged(s["q"], phs.PagedPool(s["k"], s["v"]), s["table"], s["lens"],
                                     s["max_len"], weights, out_dtype=s["dtype"],
                                     k_new=s["k_new"], v_new=s["v_new"])
    return dict(out=out, k=s["k"], v=s["v"])


def _plain_recur(s):
    c = s["case"]
    b, hk, d = c["batch"], c["kv_heads"], c["dim"]
    ids = s["ids"].long()
    state = s["state"][ids] * torch.exp(s["decay"])[:, None, None]
    state = state + s["k"].float()[..., :, None] * s["v"].float()[..., None, :]
    s["state"][ids] = state
    q = s["q"].float().view(b, hk, -1, d) * s["scale"]
    o = torch.einsum("bhgk,bhkv->bhgv", q, state).reshape(b, -1, d)
    return dict(out=o.to(s["dtype"]), state=s["state"])


def _own_recur(s):
    import paged_hybrid_sliding_gb300 as phs
    out = phs.linear_attn_decode(s["q"], s["k"], s["v"], phs.StatePool(s["state"]), s["decay"],
                                 state_ids=s["ids"], scale=s["scale"], out_dtype=s["dtype"])
    return dict(out=out, state=s["state"])


def _power(decay, n):
    """exp(decay * n) for n >= 0 and 0 for n < 0: the angle in 64 bits, [heads, *n.shape]."""
    n = n.double()
    w = torch.exp(decay.double().view(-1, *[1] * n.dim()) * n.clamp(min=0))
    return torch.where(n >= 0, w, 0.0).float()


def _plain_prompt(s):
    c = s["case"]
    b, hk, d = c["batch"], c["kv_heads"], c["dim"]
    grp, size = c["q_heads"] // hk, 64
    cu, ids = s["cu"].long(), s["ids"].long()
    lens = cu[1:] - cu[:-1]
    n = -(-s["max_len"] // size)  # chunks
    t = torch.arange(n * size, device=DEV)
    real = t < lens[:, None]
    at = torch.where(real, cu[:-1, None] + t, 0)
    mask = real[:, :, None, None]
    q = (s["q"][at].float() * s["scale"] * mask).view(b, n, size, hk, grp, d)
    k = (s["k"][at].float() * mask).view(b, n, size, hk, d)
    v = (s["v"][at].float() * mask).view(b, n, size, hk, d)
    first = torch.where(s["resume"][:, None, None, None] != 0, s["state"][ids], 0.0)
    i, ch = torch.arange(size, device=DEV), torch.arange(n, device=DEV)
    # within a chunk
    w = torch.einsum("bnihgd,bnjhd->bnhgij", q, k)
    w = w * _power(s["decay"], i[:, None] - i)[:, None]
    o = torch.einsum("bnhgij,bnjhd->bnihgd", w, v)
    # the chunks' own states, summed with their decay into the state before each chunk
    add = torch.einsum("hj,bnjhk,bnjhv->bnhkv", _power(s["decay"], size - 1 - i), k, v)
    before = torch.einsum("hnm,bmhkv->bnhkv", _power(s["decay"], size * (ch[:, None] - 1 - ch)), add)
    before = before + _power(s["decay"], size * ch).t()[None, :, :, None, None] * first[:, None]
    o = o + torch.einsum("hi,bnihgk,bnhkv->bnihgv", _power(s["decay"], i + 1), q, before)
    out = o.reshape(b, n * size, c["q_heads"], d)[real].bfloat16()
    # the state after the last token
    w = _power(s["decay"], lens[:, None] - 1 - t)  # [heads, batch, tokens]
    k = k.view(b, n * size, hk, d) * w.permute(1, 2, 0)[..., None]
    end = torch.einsum("bthk,bthv->bhkv", k, v.view(b, n * size, hk, d))
    s["state"][ids] = end + _power(s["decay"], lens).t()[:, :, None, None] * first
    return dict(out=out, state=s["state"])


def _own_prompt(s):
    import paged_hybrid_sliding_gb300 as phs
    out = phs.linear_attn_prompt(s["q"], s["k"], s["v"], s["cu"], s["max_len"],
                                 phs.StatePool(s["state"]), s["decay"], state_ids=s["ids"],
                                 resume=s["resume"], scale=s["scale"])
    return dict(out=out, state=s["state"])


_plain = dict(fork=_plain_fork, compact=_plain_compact, diff=_plain_diff, recur=_plain_recur,
              prompt=_plain_prompt)
_own = dict(fork=_own_fork, compact=_own_compact, diff=_own_diff, recur=_own_recur,
            prompt=_own_prompt)


# -------------------------------------------------------------------- work --
def work(c):
    if c["op"] == "fork":
        lens = _lens(c, c["parents"])[np.arange(c["children"]) % c["parents"]]
        page = 2 * c["layers"] * c["heads"] * PAGE * c["dim"] * 2
        # a table entry and a count read and written for each page freed and each page shared
        entries = int(_pages(lens).sum()) + int(_pages(_lens(c, c["children"])).sum())
        return dict(bytes=2 * page * int((lens % PAGE != 0).sum()) + 16 * entries, flops=0)
    if c["op"] == "compact":
        page = 2 * c["layers"] * c["heads"] * PAGE * c["dim"] * 2
        cells = c["rows"] * (int(_pages(_lens(c, c["rows"])).max()) + 3)
        return dict(bytes=2 * page * c["moves"] + 8 * cells + 12 * c["pages"], flops=0)
    if c["op"] == "diff":
        t, d = int(_lens(c, c["batch"]).sum()), c["dim"]
        rows = c["batch"] * c["heads"] * 2 * d
        return dict(bytes=t * 2 * c["value_heads"] * d * 4 + rows * (6 if c["f32"] else 4) + t // 4,
                    flops=t * c["heads"] * 2 * (2 * d + 4 * d))
    d = c["dim"]
    state = c["batch"] * c["kv_heads"] * d * d
    if c["op"] == "recur":
        io = c["batch"] * d * (c["q_heads"] * (6 if c["f32"] else 4) + 4 * c["kv_heads"])
        return dict(bytes=8 * state + io, flops=3 * state + 2 * c["batch"] * c["q_heads"] * d * d)
    t = int(_lens(c, c["batch"]).sum())
    return dict(bytes=4 * t * d * (c["q_heads"] + c["kv_heads"]) + 6 * state,
                flops=2 * t * d * d * (c["q_heads"] + c["kv_heads"]))


# ------------------------------------------------- the definitions, 64 bits --
def exact(case, seed):
    s = prepare(case, seed)
    return dict(fork=_exact_fork, compact=_exact_compact, diff=_exact_diff, recur=_exact_recur,
                prompt=_exact_prompt)[case["op"]](s)


def _exact_fork(s):
    table, lens, counts = (s[x].cpu().numpy().copy() for x in ("table", "lens", "counts"))
    for r in s["dst"].cpu().numpy():
        for p in table[r, :_pages(lens[r])]:
            counts[p] -= 1
        lens[r] = 0
    free = [p for p in range(len(counts)) if counts[p] == 0]
    for a, r in zip(s["src"].cpu().numpy(), s["dst"].cpu().numpy()):
        for j in range(_pages(lens[a])):
            p = table[a, j] if (j + 1) * PAGE <= lens[a] else free.pop(0)
            table[r, j] = p
            counts[p] += 1
        lens[r] = lens[a]
    return dict(table=table, lens=lens, counts=counts, pools=[(None, None)] * len(s["pools"]))


def _exact_compact(s):
    table, lens, counts = (s[x].cpu().numpy().copy() for x in ("table", "lens", "counts"))
    num = int((counts > 0).sum())
    page_map = np.where(counts > 0, np.arange(len(counts)), -1).astype(np.int32)
    low, high = 0, len(counts) - 1
    while True:
        while low < num and counts[low] > 0:
            low += 1
        while high >= num and counts[high] == 0:
            high -= 1
        if low >= num or high < num:
            break
        page_map[high], counts[low], counts[high] = low, counts[high], 0
        low, high = low + 1, high - 1
    for r in range(len(lens)):
        for j in range(_pages(lens[r])):
            table[r, j] = page_map[table[r, j]]
    return dict(table=table, counts=counts, page_map=page_map, num_live=np.array([num], np.int32),
                pools=[(None, None)] * len(s["pools"]))


def _exact_diff(s):
    c = s["case"]
    h, vh, d = c["heads"], c["value_heads"], c["dim"]
    rows = []
    lam = _lambda(s, torch.float64)
    for r, n in enumerate(s["lens"].tolist()):
        at = s["table"][r, :_pages(n)].long()
        k = s["k"][at].transpose(1, 2).reshape(-1, 2 * vh, d)[:n].double()
        v = s["v"][at].transpose(1, 2).reshape(-1, vh, 2 * d)[:n].double()
        if c["append"]:
            k[n - 1] = s["k_new"][r].double()
            v[n - 1] = s["v_new"][r].double().reshape(vh, 2 * d)
        for i in range(h):
            j = i // (h // vh)
            maps = [torch.softmax(k[:, 2 * j + m] @ s["q"][r, 2 * i + m].double() / math.sqrt(d), 0)
                    for m in (0, 1)]
            o = (maps[0] - lam * maps[1]) @ v[:, j]
            if s["norm"] is not None:
                o = o / torch.sqrt((o @ o) / (2 * d) + s["eps"]) * s["norm"].double()
                o = o * (1 - s["lam_init"])
            rows.append(o)
    return dict(out=torch.stack(rows).view(c["batch"], h, 2 * d), k=None, v=None)


def _step(state, decay, k, v, q):
    """One token of the recurrence: state [.., dk, dv], k [.., dk], v [.., dv], q [.., g, dk]."""
    state = state * decay + k.unsqueeze(-1) * v.unsqueeze(-2)
    return state, q @ state


def _exact_recur(s):
    c = s["case"]
    ids = s["ids"].long()
    q = s["q"].double().view(c["batch"], c["kv_heads"], -1, c["dim"]) * s["scale"]
    new, o = _step(s["state"][ids].double(), torch.exp(s["decay"].double())[:, None, None],
                   s["k"].double(), s["v"].double(), q)
    state = s["state"].double()
    state[ids] = new
    return dict(out=o.reshape(c["batch"], -1, c["dim"]), state=state)


def _exact_prompt(s):
    c = s["case"]
    b, hk, d = c["batch"], c["kv_heads"], c["dim"]
    if b * hk * d * d * s["max_len"] > 6e10:
        return None
    cu, ids = s["cu"].long(), s["ids"].long()
    decay = torch.exp(s["decay"].double())[:, None, None]
    state = s["state"].double()
    now = state[ids] * (s["resume"] != 0)[:, None, None, None]
    out = torch.zeros(s["q"].shape[0], hk, c["q_heads"] // hk, d, dtype=torch.float64, device=DEV)
    for t, live in enumerate(_live_rows(cu, s["max_len"])):
        at = cu[live] + t
        new, out[at] = _step(now[live], decay, s["k"][at].double(), s["v"][at].double(),
                             s["q"][at].double().view(len(at), hk, -1, d) * s["scale"])
        now[live] = new
    state[ids] = now
    return dict(out=out.view(-1, c["q_heads"], d), state=state)


def _live_rows(cu, most):
    """For each position the requests that have a token there."""
    lens = (cu[1:] - cu[:-1]).tolist()
    for t in range(most):
        yield torch.tensor([r for r, n in enumerate(lens) if n > t], device=DEV)
