"""The operators of a prompt's way into a paged KV cache, as measured cases.

Before a request can be drafted for, the target model runs over its prompt: all at
once, or in chunks beside other requests' rows, and several continuations of one
prompt share its pages.  What that needs beside the model's own products:

  rope     norm of every head of the queries and keys, the rotation by position, and
           the keys and values into their cache slots
  attn     attention of a chunk of new rows of each request over its cached tokens
           and the chunk's own earlier rows
  fork     continuations of prompts: full pages shared, the last one copied; and their
           end, when pages that nobody holds any more are free again
  squeeze  the pages in use moved to the lowest numbers, so that the rest can go back

Each case runs in its plain form (elementary torch operations in 32 bits) or,
with `own` set, through the framework's entry points.
"""
import math
import random

import torch

own = False

FP8_MAX = 448.0
EPS = 1e-6


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # four requests' next tokens: the call's latency
        dict(name="rope_tokens", op="rope", R=4, n_lo=1, n_hi=1, ctx_lo=100, ctx_hi=3000, Hq=32,
             Hkv=8, D=128, rot=128, pairs=False, norm=True, base=1e6, page=64, fp8=False, pad=0),
        # eight prompts of two thousand tokens, all heads rotated as halves
        dict(name="rope_prompts", op="rope", R=8, n_lo=2048, n_hi=2048, ctx_lo=1, ctx_hi=64, Hq=32,
             Hkv=8, D=128, rot=128, pairs=False, norm=True, base=1e6, page=32, fp8=False, pad=0),
        # ragged chunks far into long contexts, half of each head rotated in pairs, an 8-bit
        # cache, rows of padding behind the last request (a launch of fixed size)
        dict(name="rope_chunks_fp8", op="rope", R=21, n_lo=3, n_hi=900, ctx_lo=5, ctx_hi=1000000,
             Hq=20, Hkv=4, D=128, rot=64, pairs=True, norm=True, base=1e4, page=16, fp8=True,
             pad=77),
        # a short prompt alone: latency
        dict(name="attn_short", op="attn", R=1, n_lo=100, n_hi=100, ctx_lo=0, ctx_hi=0, Hq=8,
             Hkv=2, D=64, page=16, fp8=False, fused=True),
        # one long prompt at once
        dict(name="attn_prompt", op="attn", R=1, n_lo=8192, n_hi=8192, ctx_lo=0, ctx_hi=0, Hq=32,
             Hkv=8, D=128, page=64, fp8=False, fused=True),
        # a serving step: next tokens and chunks of prompts together, ragged, five query
        # heads to a KV head
        dict(name="attn_mixed", op="attn", R=12, n_lo=1, n_hi=1500, ctx_lo=3, ctx_hi=6000, Hq=40,
             Hkv=8, D=128, page=16, fp8=False, fused=True),
        # the next chunks of two long prompts in an 8-bit cache
        dict(name="attn_long_fp8", op="attn", R=2, n_lo=500, n_hi=512, ctx_lo=40000, ctx_hi=50000,
             Hq=32, Hkv=8, D=128, page=128, fp8=True, fused=False),
        # the largest: second chunks of eight prompts
        dict(name="attn_chunks", op="attn", R=8, n_lo=4096, n_hi=4096, ctx_lo=4096, ctx_hi=4096,
             Hq=32, Hkv=8, D=128, page=32, fp8=False, fused=True),
        # three samples of one prompt
        dict(name="fork_samples", op="fork", R=8, sources=1, forks=3, ctx_lo=333, ctx_hi=333,
             Hkv=8, D=128, page=16, fp8=False),
        # fifteen samples of each of 32 prompts
        dict(name="fork_batch", op="fork", R=1024, sources=32, forks=480, ctx_lo=100, ctx_hi=5000,
             Hkv=8, D=128, page=64, fp8=False),
        # a small cache, a few of whose requests have left
        dict(name="squeeze_small", op="squeeze", R=8, pages=96, held=0.5, Hkv=2, D=64, page=16,
             fp8=True),
        # half of a cache of a gigabyte is free, in holes
        dict(name="squeeze_batch", op="squeeze", R=300, pages=8000, held=0.5, Hkv=8, D=128,
             page=32, fp8=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "attn", "attn", "attn", "attn", "fork", "squeeze"])
    c = dict(op=op)
    if op in ("rope", "attn"):
        c.update(R=_log_int(rng, 1, 48), n_lo=_log_int(rng, 1, 512))
        c.update(n_hi=_log_int(rng, c["n_lo"], 4096), ctx_lo=_log_int(rng, 1, 2048) - 1)
        Hkv = rng.choice([1, 2, 4, 8])
        c.update(Hq=Hkv * rng.choice([1, 2, 4, 5, 8]), Hkv=Hkv, D=rng.choice([64, 128]),
                 page=rng.choice([16, 32, 64, 128]), fp8=rng.random() < 0.4)
    if op == "rope":
        c.update(rot=rng.choice([16, 32, 64, c["D"], c["D"]]), pairs=rng.random() < 0.5,
                 norm=rng.random() < 0.7, base=rng.choice([1e4, 5e5, 1e6]),
                 ctx_hi=_log_int(rng, c["ctx_lo"] + 1, 2000000), pad=rng.choice([0, 0, 1, 50]))
        while work(c)["bytes"] > 6e8:
            c["R"], c["n_hi"] = max(1, c["R"] // 2), max(c["n_lo"], c["n_hi"] * 2 // 3)
    elif op == "attn":
        c.update(ctx_hi=_log_int(rng, c["ctx_lo"] + 1, 65536), fused=rng.random() < 0.6)
        # no dearer than the largest listed case, and the plain form's padded scores stay small
        while True:
            long = c["ctx_hi"] + c["n_hi"]
            scores = 4.0 * c["R"] * c["Hq"] * c["n_hi"] * long
            padded = 4.0 * c["R"] * c["Hkv"] * c["D"] * long
            if scores <= 3.5e10 and padded <= 8e9 and work(c)["flops"] <= 3.2e12:
                break
            if c["R"] > 4:
                c["R"] = c["R"] * 2 // 3
            elif c["n_hi"] > 2 * c["n_lo"]:
                c["n_hi"] = c["n_hi"] * 2 // 3
            else:
                c["ctx_hi"] = max(c["ctx_lo"], c["ctx_hi"] * 2 // 3)
                c["n_lo"] = max(1, c["n_lo"] * 2 // 3)
                c["n_hi"] = max(c["n_lo"], c["n_hi"] * 2 // 3)
    elif op == "fork":
        c.update(R=_log_int(rng, 2, 1024), Hkv=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 128]),
                 page=rng.choice([16, 32, 64, 128]), fp8=rng.random() < 0.4)
        c.update(sources=_log_int(rng, 1, max(1, c["R"] // 4)))
        c.update(forks=_log_int(rng, 1, c["R"] - c["sources"]), ctx_lo=_log_int(rng, 1, 500))
        c.update(ctx_hi=_log_int(rng, c["ctx_lo"], min(5000, max(c["ctx_lo"], 100000 // c["sources"]))))
    else:
        c.update(R=_log_int(rng, 1, 512), pages=_log_int(rng, 16, 8000),
                 held=round(rng.uniform(0.05, 0.95), 2), Hkv=rng.choice([1, 2, 4, 8]),
                 D=rng.choice([64, 128]), page=rng.choice([16, 32, 64]), fp8=rng.random() < 0.4)
        # a cache of the largest listed one's size at most
        each = c["page"] * c["Hkv"] * c["D"] * 4
        c["pages"] = min(c["pages"], int(1.04e9 / each))
    return c


def _spread(lo, hi, n):
    """n lengths from lo to hi, evenly over their logarithm, in order."""
    return [int(round((lo + 1) * ((hi + 1) / (lo + 1)) ** ((i + 0.5) / n))) - 1 for i in range(n)]


def _requests(c):
    """The batch's (context, new rows): short contexts with few and with many rows."""
    ctx, rows = _spread(c["ctx_lo"], c["ctx_hi"], c["R"]), _spread(c["n_lo"], c["n_hi"], c["R"])
    random.Random(c["R"]).shuffle(rows)
    return list(zip(ctx, rows))


def _prompts(c):
    """The sources' lengths, and how many forks each has."""
    n = c["sources"]
    return _spread(c["ctx_lo"], c["ctx_hi"], n), [len(range(i, c["forks"], n)) for i in range(n)]


def work(case):
    """Bytes and operations of one pass."""
    c, op = case, case["op"]
    size = 1 if c["fp8"] else 2
    vec = 2 * c["Hkv"] * c["D"]  # K and V values of one token
    if op == "rope":  # heads in, queries out, keys and values into the cache
        rows = sum(n for _, n in _requests(c))
        return {"bytes": rows * (c["Hq"] * c["D"] * 4.0 + vec * (2 + size) + 12), "flops": 0}
    if op == "attn":  # each cached token once, queries in, results and their log-sums out
        both = _requests(c)
        tokens, rows = sum(x + n for x, n in both), sum(n for _, n in both)
        seen = sum(n * x + n * (n + 1) / 2 for x, n in both)
        return {"bytes": tokens * vec * size + rows * c["Hq"] * (c["D"] * 4.0 + 4)
                + 4.0 * tokens / c["page"], "flops": 4.0 * c["Hq"] * c["D"] * seen}
    if op == "fork":  # tables of the forks written and read again, the last pages copied
        ctx, forks = _prompts(c)
        pages = sum(-(-x // c["page"]) * n for x, n in zip(ctx, forks))
        tail = sum(x % c["page"] * n for x, n in zip(ctx, forks))
        return {"bytes": 2.0 * tail * vec * size + 20.0 * pages + 32.0 * c["forks"], "flops": 0}
    used = _used(c)
    moved = used * (c["pages"] - used) / c["pages"]  # as the holes lie anywhere
    return {"bytes": 2.0 * moved * c["page"] * vec * size + 24.0 * c["pages"], "flops": 0}


def _used(c):
    return max(1, min(c["pages"] - 1, int(c["pages"] * c["held"])))


# ----------------------------------------------------------------- inputs ----

def _order(c, seed):
    """The requests of the batch in this seed's order."""
    both = _requests(c)
    random.Random(seed).shuffle(both)
    return both


def _deal(order, pages, max_pages):
    """Block table whose rows hold `pages` of `order` in turn; -1 behind them."""
    first = pages.cumsum(0) - pages
    col = torch.arange(max_pages, device="cuda")
    at = (first[:, None] + col).clamp(max=order.numel() - 1)
    return torch.where(col < pages[:, None], order[at], -1).to(torch.int32).contiguous()


def _cache(c, n_pages, g):
    shape = (n_pages, c["page"], c["Hkv"], c["D"])
    out = {}
    for x in ("k", "v"):
        t = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
        if c["fp8"]:
            scale = 0.01 + 0.01 * torch.rand((c["Hkv"],), generator=g, device="cuda")
            t = (t.float() / scale[:, None]).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
            out[x + "_scale"] = scale
        out[x + "c"] = t
    return out


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(c=c)
    if c["op"] in ("rope", "attn"):
        return _prepare_rows(c, s, g, seed)
    if c["op"] == "fork":
        return _prepare_fork(c, s, g)
    # squeeze: requests of about equal size hold `used` pages anywhere in the cache, every
    # third one's first pages shared with the request before it
    n, used = c["pages"], _used(c)
    order = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
    R = min(c["R"], used)
    at = torch.arange(R, device="cuda")
    held = (used * (at + 1)) // R - (used * at) // R
    table = _deal(order, held, int(held.max()))
    shared = ((at % 3 == 2) & (at > 0)).nonzero().flatten()
    take = torch.minimum(held[shared - 1], held[shared])
    pages = held + held.new_zeros(R).index_put((shared,), take)
    wide = torch.full((R, 2 * table.shape[1]), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    col = torch.arange(wide.shape[1], device="cuda")
    for_shared = torch.where(col < take[:, None], wide[shared - 1],
                             wide[shared].gather(1, (col - take[:, None]).clamp(min=0)))
    wide[shared] = for_shared
    refs = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    flat = wide[col < pages[:, None]].long()
    refs.index_add_(0, flat, torch.ones_like(flat, dtype=torch.int32))
    s["refs"] = refs.clamp(min=0)
    s["table"], s["held"] = wide, pages.to(torch.int32)
    s["free"] = torch.cat([order[used:], order[:used]]).contiguous()
    s["n_free"] = torch.tensor([n - used], dtype=torch.int32, device="cuda")
    s.update(_cache(c, n, g))
    return s


def _prepare_rows(c, s, g, seed):
    both = _order(c, seed)
    R, ps, Hq, Hkv, D = c["R"], c["page"], c["Hq"], c["Hkv"], c["D"]
    ctx, n = (torch.tensor(x, device="cuda") for x in zip(*both))
    start = torch.cat([n.new_zeros(1), n.cumsum(0)])
    rows = int(sum(x for _, x in both))
    cap = rows + c.get("pad", 0)
    req = torch.repeat_interleave(torch.arange(R, device="cuda"), n)
    position = ctx[req] + torch.arange(rows, device="cuda") - start[req]
    randn = lambda *k: torch.randn(k, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    if c["op"] == "rope":
        # slots: pages of their own for the new rows, in any order
        pages = (ctx + n - 1) // ps - ctx // ps + 1
        n_pages = sum((x + m - 1) // ps - x // ps + 1 for x, m in both) + 5
        table = _deal(torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32), pages,
                      max((x + m - 1) // ps - x // ps + 1 for x, m in both))
        slot = table[req, position // ps - ctx[req] // ps].long() * ps + position % ps
        fill = torch.full((cap - rows,), -1, device="cuda")
        s["position"] = torch.cat([position, fill]).to(torch.int32)
        s["slot"] = torch.cat([slot, fill])
        qkv = randn(cap, Hq + 2 * Hkv, D)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        s["q_weight"] = s["k_weight"] = None
        if c["norm"]:
            s["q_weight"], s["k_weight"] = (1 + 0.2 * randn(D)).clone(), (1 + 0.2 * randn(D)).clone()
        i = torch.arange(c["rot"] // 2, device="cuda", dtype=torch.float64)
        s["inv_freq"] = c["base"] ** (-2 * i / c["rot"])
        s["q_out"] = torch.zeros((cap, Hq, D), dtype=torch.bfloat16, device="cuda")
        s.update(_cache(c, n_pages, g))
        return s
    total = ctx + n
    pages = (total + ps - 1) // ps
    n_pages = sum(-(-(x + m) // ps) for x, m in both) + 8
    s["lengths"] = both
    s["max_pages"] = max(-(-(x + m) // ps) for x, m in both)
    s["max_rows"] = max(m for _, m in both)
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    s["table"] = _deal(order, pages, s["max_pages"])
    s["ctx"], s["row_start"] = ctx.to(torch.int32), start.to(torch.int32)
    s.update(_cache(c, n_pages, g))
    wide = Hq + (2 * Hkv if c["fused"] else 0)
    s["q"] = (1.5 * randn(rows, wide, D))[:, :Hq]
    s["out"] = torch.zeros((rows, Hq, D), dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.zeros((rows, Hq), dtype=torch.float32, device="cuda")
    return s


def _prepare_fork(c, s, g):
    R, ps, n = c["R"], c["page"], c["sources"]
    lengths, forks = _prompts(c)
    place = torch.randperm(R, generator=g, device="cuda")
    ctx = torch.full((R,), -1, device="cuda")
    ctx[place[:n]] = torch.tensor(lengths, device="cuda")
    held = torch.where(ctx >= 0, (ctx + ps) // ps, 0)  # a page ahead where the last one is full
    n_pages = sum((x + ps) // ps for x in lengths) + c["forks"] + 4
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    s["table"] = _deal(order, held, max((x + ps) // ps for x in lengths))
    used = sum((x + ps) // ps for x in lengths)
    s["free"] = torch.cat([order[used:], order[:used]]).contiguous()
    s["n_free"] = torch.tensor([n_pages - used], dtype=torch.int32, device="cuda")
    s["ctx"], s["held"] = ctx.to(torch.int32), held.to(torch.int32)
    s["refs"] = torch.zeros((n_pages,), dtype=torch.int32, device="cuda")
    # fork i goes from prompt i mod n to the free place of the i-th highest number, so that
    # what a pass takes off the stack comes back in the order in which it lay there
    s["source"] = place[torch.arange(c["forks"], device="cuda") % n].to(torch.int32)
    s["target"] = place[n:n + c["forks"]].sort(descending=True).values.to(torch.int32)
    s["place"] = s["target"].long()
    s.update(_cache(c, n_pages, g))
    new = lambda: torch.full((c["forks"],), -7, dtype=torch.int32, device="cuda")  # noqa: E731
    s["from"], s["to"], s["tokens"] = new(), new(), new()
    return s


# ------------------------------------------------------------ plain forms ----

def _rotated(x, weight, cos, sin, rot, pairs):
    """x [rows, heads, D] in f32: normalised, then the first `rot` values turned."""
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    if pairs:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([a, b], -1).flatten(-2) if pairs else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def plain_rope(s):
    c = s["c"]
    ps = c["page"]
    angle = s["position"].double()[:, None, None] * s["inv_freq"]
    cos, sin = angle.cos().float(), angle.sin().float()
    q = _rotated(s["q"].float(), s["q_weight"], cos, sin, c["rot"], c["pairs"])
    k = _rotated(s["k"].float(), s["k_weight"], cos, sin, c["rot"], c["pairs"])
    there = s["position"] >= 0
    q_out = torch.where(there[:, None, None], q.to(torch.bfloat16), s["q_out"])
    # rows of padding write where the last row does, with that row's values
    keep = s["slot"] >= 0
    row = torch.where(keep, torch.arange(keep.numel(), device="cuda"), keep.sum() - 1)
    page, at = s["slot"][row] // ps, s["slot"][row] % ps
    raw = (lambda t: t.view(torch.uint8)) if c["fp8"] else (lambda t: t)
    raw(s["kc"])[page, at] = raw(_stored(k, s.get("k_scale")))[row]
    raw(s["vc"])[page, at] = raw(_stored(s["v"].float(), s.get("v_scale")))[row]
    return q_out, s["kc"], s["vc"]


def _stored(x, scale):
    if scale is None:
        return x.to(torch.bfloat16)
    return (x / scale[:, None]).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)


def plain_attn(s):
    """Every request's rows and tokens padded to the longest one's."""
    c = s["c"]
    R, W, H, D = c["R"], s["max_rows"], c["Hkv"], c["D"]
    rep, L, rows = c["Hq"] // H, s["max_pages"] * c["page"], s["q"].shape[0]
    start = s["row_start"].long()
    n = start[1:] - start[:-1]
    i = torch.arange(W, device="cuda")
    row_ok = i < n[:, None]
    row = torch.where(row_ok, start[:-1, None] + i, 0)
    pos = torch.arange(L, device="cuda")
    last = s["ctx"].long()[:, None] + i                       # a row's own position [R, W]
    inside = pos < (s["ctx"].long() + n)[:, None]
    table = s["table"].long().clamp(min=0)

    def gathered(x, scale):  # [R, H, L, D] in f32, zero past the request's end
        raw = x.view(torch.uint8)[table].view(x.dtype) if c["fp8"] else x[table]
        y = raw.view(R, L, H, D).float()
        if scale is not None:
            y = y * scale[:, None]
        return y.masked_fill_(~inside[:, :, None, None], 0.0).permute(0, 2, 1, 3)

    q = s["q"][row].float().view(R, W, H, rep, D).permute(0, 2, 3, 1, 4)       # [R, H, rep, W, D]
    score = q.reshape(R, H, rep * W, D) @ gathered(s["kc"], s.get("k_scale")).transpose(2, 3)
    score = score.mul_(1 / math.sqrt(D)).view(R, H, rep, W, L)
    score.masked_fill_((pos > last[..., None])[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(R, H, rep * W, L) @ gathered(s["vc"], s.get("v_scale"))).view(R, H, rep, W, D)
    o, lse = o / total, top + torch.log(total)
    back = lambda t: t.permute(0, 3, 1, 2, 4).reshape(R * W, H * rep, -1)  # noqa: E731
    to = torch.where(row_ok, row, rows).reshape(-1)  # padded rows go to a row of their own
    out = torch.zeros((rows + 1, c["Hq"], D), dtype=torch.bfloat16, device="cuda")
    out[to] = back(o).to(torch.bfloat16)
    lse_out = torch.zeros((rows + 1, c["Hq"]), device="cuda")
    lse_out[to] = back(lse).squeeze(-1)
    return out[:-1], lse_out[:-1]


def plain_fork(s):
    c = s["c"]
    ps, pages, width = c["page"], s["free"].numel(), s["table"].shape[1]
    col = torch.arange(width, device="cuda")
    src, dst = s["source"].long(), s["target"].long()
    # the forks: full pages shared, a page off the stack for what is left
    tokens = s["ctx"].long()[src]
    full, tail = tokens // ps, tokens % ps
    need = (tail > 0).long()
    top = s["n_free"].long()
    fresh = s["free"].long()[top - need.cumsum(0)]
    last = s["table"][src, full.clamp(max=width - 1)].long()
    shared = col < full[:, None]
    row = torch.where(shared, s["table"][src].long(), s["table"][dst].long())
    row = torch.where((col == full[:, None]) & (need > 0)[:, None], fresh[:, None], row)
    table = s["table"].clone()
    table[dst] = row.to(torch.int32)
    holders = s["refs"].long().new_zeros(pages + 1)
    mine = torch.where(shared, row, pages)
    holders.index_add_(0, mine.flatten(), torch.ones_like(mine.flatten()))
    # the last pages' tokens (what is no copy stays where it is)
    raw = (lambda t: t.view(torch.uint8)) if c["fp8"] else (lambda t: t)
    at = torch.arange(ps, device="cuda")
    to_page = torch.where(need > 0, fresh, last)[:, None].expand(-1, ps)
    from_page = torch.where(at < tail[:, None], last[:, None], to_page)
    for_k, for_v = raw(s["kc"])[from_page, at], raw(s["vc"])[from_page, at]
    raw(s["kc"])[to_page, at] = for_k
    raw(s["vc"])[to_page, at] = for_v
    # the end of the forks: each page goes back with the last of its holders, request by request
    order = torch.argsort(dst)
    leaves = (col < (full + need)[:, None])[order]
    page = torch.where(leaves, row[order], pages).flatten()
    count = page.new_zeros(pages + 1).index_add_(0, page, torch.ones_like(page))
    where = torch.full_like(count, -1).scatter_reduce_(0, page, torch.arange(page.numel(), device="cuda"),
                                                       "amax")
    refs = torch.cat([s["refs"].long(), s["refs"].new_zeros(1).long()]) + holders
    gone = (count == refs + 1)[page] & (page < pages) & (where[page] == torch.arange(page.numel(), device="cuda"))
    rest = (refs - count).clamp(min=0)[:-1]
    free = torch.cat([s["free"].long(), top])
    place = top - need.sum() + gone.long().cumsum(0) - 1
    free[torch.where(gone, place, pages)] = page
    held = s["held"].clone()
    held[dst] = 0
    ctx = s["ctx"].clone()
    ctx[dst] = -1
    i32 = lambda t: t.to(torch.int32)  # noqa: E731
    return dict(table=table, held=held, ctx=ctx, refs=i32(rest), free=i32(free[:-1]),
                n_free=i32(top - need.sum() + gone.sum()), copy_from=i32(torch.where(need > 0, last, -1)),
                copy_to=i32(torch.where(need > 0, fresh, -1)), copy_tokens=i32(tail),
                k=s["kc"], v=s["vc"])


def plain_squeeze(s):
    c = s["c"]
    n = c["pages"]
    page = torch.arange(n, device="cuda")
    place = torch.arange(n, device="cuda")
    is_free = torch.zeros((n,), dtype=torch.bool, device="cuda")
    is_free = is_free.index_put((s["free"].long(),), place < s["n_free"])
    used = n - s["n_free"].long()
    # the used pages past the first `used` ones, in order, into the free ones below, in order
    out, into = ~is_free & (page >= used), is_free & (page < used)
    moves = out.sum()
    by = torch.full((n + 1,), -1, dtype=torch.long, device="cuda")
    goes = by.index_put((torch.where(out, out.cumsum(0) - 1, n),), page)[:n]
    takes = by.index_put((torch.where(into, into.cumsum(0) - 1, n),), page)[:n]
    valid = page < moves
    goes, takes = torch.where(valid, goes, -1), torch.where(valid, takes, -1)
    new = torch.where(is_free, -1, page)
    new = torch.cat([new, new[:1]]).index_put((torch.where(valid, goes, n),), takes)[:n]
    col = torch.arange(s["table"].shape[1], device="cuda")
    table = torch.where(col < s["held"][:, None], new[s["table"].long().clamp(min=0)], s["table"].long())
    refs = torch.zeros((n + 1,), dtype=torch.long, device="cuda")
    refs = refs.index_put((torch.where(new >= 0, new, n),), s["refs"].long())[:n]
    free = torch.where(place < s["n_free"], n - 1 - place, s["free"].long())
    raw = (lambda t: t.view(torch.uint8)) if c["fp8"] else (lambda t: t)
    half = n // 2
    # what is no move copies the lowest used page of the squeezed cache onto itself
    a = torch.where(valid, goes, takes[:1].clamp(min=0))[:half]
    b = torch.where(valid, takes, takes[:1].clamp(min=0))[:half]
    a = torch.where(valid[:half], a, torch.where(moves > 0, goes[:1], 0))
    for_k, for_v = raw(s["kc"])[a], raw(s["vc"])[a]
    raw(s["kc"])[b] = for_k
    raw(s["vc"])[b] = for_v
    i32 = lambda t: t.to(torch.int32)  # noqa: E731
    return dict(table=i32(table), refs=i32(refs), free=i32(free), new=i32(new),
                move_from=i32(goes[:half]), move_to=i32(takes[:half]), moves=i32(moves.view(1)),
                k=s["kc"], v=s["vc"])


PLAIN = dict(rope=plain_rope, attn=plain_attn, fork=plain_fork, squeeze=plain_squeeze)


# -------------------------------------------------- the framework's calls ----

def _own_cache(s):
    import speculative_decoding_draft_02_gb300 as dsp
    if "cache" not in s:
        s["cache"] = dsp.KVCache(s["kc"], s["vc"], s.get("k_scale"), s.get("v_scale"))
    return dsp, s["cache"]


def own_rope(s):
    dsp, cache = _own_cache(s)
    if "rotary" not in s:
        s["rotary"] = dsp.Rotary(s["inv_freq"], pairs=s["c"]["pairs"])
    dsp.dspark_rope_append(cache, s["q"], s["k"], s["v"], s["position"], s["slot"], s["rotary"],
                           s["q_out"], s["q_weight"], s["k_weight"], EPS)
    return s["q_out"], s["kc"], s["vc"]


def own_attn(s):
    dsp, cache = _own_cache(s)
    c = s["c"]
    if "ws" not in s:
        s["ws"] = dsp.workspace(dsp.dspark_chunk_attention_workspace_bytes(
            cache, c["R"], c["Hq"], s["max_rows"]))
    dsp.dspark_chunk_attention(cache, s["q"], s["ctx"], s["row_start"], s["table"], s["max_rows"],
                               1 / math.sqrt(c["D"]), s["out"], s["lse"], s["ws"])
    return s["out"], s["lse"]


def own_fork(s):
    dsp, cache = _own_cache(s)
    dsp.dspark_kv_fork(s["source"], s["target"], s["c"]["page"], s["ctx"], s["held"], s["n_free"],
                       s["free"], s["table"], s["refs"], s["from"], s["to"], s["tokens"])
    dsp.dspark_kv_copy(cache, s["from"], s["to"], s["tokens"])
    s["ctx"].index_fill_(0, s["place"], -1)
    dsp.dspark_kv_release(s["ctx"], s["held"], s["n_free"], s["free"], s["table"], s["refs"])
    return dict(table=s["table"], held=s["held"], ctx=s["ctx"], refs=s["refs"], free=s["free"],
                n_free=s["n_free"], copy_from=s["from"], copy_to=s["to"], copy_tokens=s["tokens"],
                k=s["kc"], v=s["vc"])


def own_squeeze(s):
    dsp, cache = _own_cache(s)
    if "o" not in s:
        new = lambda *n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
        n = s["c"]["pages"]
        s["o"] = dict(table=torch.empty_like(s["table"]), refs=new(n), free=new(n), new=new(n),
                      move_from=new(n // 2), move_to=new(n // 2), moves=new(1))
    o = s["o"]
    dsp.dspark_kv_squeeze(s["held"], s["n_free"], s["free"], s["table"], s["refs"], o["free"],
                          o["table"], o["refs"], o["new"], o["move_from"], o["move_to"],
                          o["moves"])
    dsp.dspark_kv_copy(cache, o["move_from"], o["move_to"])
    return dict(o, k=s["kc"], v=s["vc"])


OWN = dict(rope=own_rope, attn=own_attn, fork=own_fork, squeeze=own_squeeze)


def run(state):
    return (OWN if own else PLAIN)[state["c"]["op"]](state)


# ------------------------------------------------------------ in 64 bits ----

def exact(case, seed):
    c = case
    if c["op"] == "rope":
        return _exact_rope(c, prepare(c, seed))
    if c["op"] == "attn":
        return _exact_attn(c, prepare(c, seed))
    return None  # whole numbers, and copies of stored values


def _exact_rope(c, s):
    """As products with unit complex numbers, one position at a time."""
    rows = int((s["position"] >= 0).sum())
    unit = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       s["position"][:rows].double()[:, None] * s["inv_freq"])[:, None]

    def turned(x, weight):
        x = x[:rows].double()
        if weight is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / c["D"] + EPS).sqrt() * weight.double()
        half = c["rot"] // 2
        head = x[..., :c["rot"]]
        two = head.unflatten(-1, (half, 2)) if c["pairs"] else head.unflatten(-1, (2, half)).mT
        z = torch.view_as_real(torch.view_as_complex(two.contiguous()) * unit)
        x[..., :c["rot"]] = (z if c["pairs"] else z.mT).flatten(-2)
        return x

    q_out = s["q_out"].double()
    q_out[:rows] = turned(s["q"], s["q_weight"])
    caches = []
    for x, new in (("k", turned(s["k"], s["k_weight"])), ("v", s["v"][:rows].double())):
        cache = s[x + "c"].double().view(-1, c["Hkv"], c["D"])
        if c["fp8"]:
            new = (new / s[x + "_scale"].double()[:, None]).clamp(-FP8_MAX, FP8_MAX)
        cache[s["slot"][:rows]] = new
        caches.append(cache.view(s["kc"].shape))
    return q_out, *caches


def _exact_attn(c, s):
    """Request by request and KV head by KV head, each with its own tokens alone."""
    H, D, Hq, ps = c["Hkv"], c["D"], c["Hq"], c["page"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    row = 0
    for r, (ctx, n) in enumerate(s["lengths"]):
        pages = s["table"][r, :-(-(ctx + n) // ps)].long()
        hide = torch.ones((n, ctx + n), dtype=torch.bool, device="cuda").triu_(ctx + 1)
        for h in range(H):
            k, v = (torch.stack([s[x][int(p), :, h].double() for p in pages]) if c["fp8"]
                    else s[x][pages, :, h].double() for x in ("kc", "vc"))
            k, v = k.reshape(-1, D)[:ctx + n], v.reshape(-1, D)[:ctx + n]
            if c["fp8"]:
                k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
            for q in range(h * Hq // H, (h + 1) * Hq // H):
                z = s["q"][row:row + n, q].double() @ k.T / math.sqrt(D)
                z.masked_fill_(hide, -math.inf)
                lse[row:row + n, q] = torch.logsumexp(z, -1)
                out[row:row + n, q] = torch.softmax(z, -1) @ v
        row += n
    return out, lse
