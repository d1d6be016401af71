"""The operators of a verification round over a paged KV cache, as measured cases.

Between the schedule (admitted draft lengths) and the verification, the target
model runs over each request's anchor and admitted drafts.  The operators here
are what that step needs beside the model's own products:

  plan     row offsets, pages, slots, positions and ancestor masks of the rows
  append   the rows' K and V into their cache slots (bf16, or e4m3 with a scale per head)
  attn     attention of the drafted tree over the cache
  accept   the path of the tree that the target's choices confirm
  compact  the rows' K and V appended, then the accepted path moved together

Each case runs in its plain form (elementary torch operations in 32 bits) or,
with `own` set, through the framework's entry points.
"""
import math

import torch

own = False

FP8_MAX = 448.0


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # one small batch's chains: the call's latency
        dict(name="plan_tiny_chain", op="plan", R=4, gamma=5, tree=False, ragged=True, page=16,
             leave=False, ctx_lo=1, ctx_hi=256),
        # the scheduler's stress concurrency, trees of 32 nodes with ragged admission, some
        # requests finished since the last round
        dict(name="plan_stress_tree", op="plan", R=1024, gamma=31, tree=True, ragged=True, page=16,
             leave=True, ctx_lo=16, ctx_hi=8192),
        # one round's rows of 256 requests at draft length 5
        dict(name="append_round", op="append", R=256, gamma=5, ragged=True, Hkv=8, D=128, page=64,
             fp8=False, fused=True, ctx_lo=64, ctx_hi=2048),
        # a prompt-sized write into an 8-bit cache
        dict(name="append_prompts_fp8", op="append", R=8, gamma=2047, ragged=False, Hkv=8, D=128,
             page=32, fp8=True, fused=True, ctx_lo=1, ctx_hi=64),
        # one request, one new token, a short context: plain decoding, latency
        dict(name="attn_single", op="attn", R=1, gamma=0, tree=False, ragged=False, Hq=32, Hkv=8,
             D=128, page=16, fp8=False, fused=False, ctx_lo=1000, ctx_hi=1000),
        # 256 requests, admitted chains of 1 to 6 rows, contexts over two decades: streaming
        dict(name="attn_chains", op="attn", R=256, gamma=5, tree=False, ragged=True, Hq=32, Hkv=8,
             D=128, page=64, fp8=False, fused=True, ctx_lo=64, ctx_hi=8192),
        # 64 requests with full trees of 64 nodes: 256 query rows for each KV head
        dict(name="attn_trees", op="attn", R=64, gamma=63, tree=True, ragged=False, Hq=32, Hkv=8,
             D=128, page=16, fp8=False, fused=True, ctx_lo=512, ctx_hi=4096),
        # four long contexts in an 8-bit cache: work split along the context
        dict(name="attn_long_fp8", op="attn", R=4, gamma=8, tree=False, ragged=False, Hq=32, Hkv=8,
             D=128, page=128, fp8=True, fused=True, ctx_lo=32768, ctx_hi=131072),
        # one request's chain of eight drafts
        dict(name="accept_chain", op="accept", R=1, gamma=8, tree=False, ragged=False, match=0.8),
        # the stress concurrency with trees of 64 nodes
        dict(name="accept_stress_tree", op="accept", R=1024, gamma=63, tree=True, ragged=True,
             match=0.7),
        # a small batch's trees
        dict(name="compact_small", op="compact", R=4, gamma=15, tree=True, ragged=False, Hkv=8,
             D=128, page=16, fp8=False, match=0.8, ctx_lo=100, ctx_hi=300),
        # 256 trees of 32 nodes
        dict(name="compact_batch", op="compact", R=256, gamma=31, tree=True, ragged=False, Hkv=8,
             D=128, page=32, fp8=False, match=0.8, ctx_lo=64, ctx_hi=512),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "attn", "attn", "attn", "accept", "compact"])
    c = dict(op=op)
    if op == "plan":
        c.update(R=_log_int(rng, 1, 1024), gamma=_log_int(rng, 1, 31), tree=rng.random() < 0.5,
                 ragged=rng.random() < 0.7, page=rng.choice([16, 32, 64, 128]),
                 leave=rng.random() < 0.5)
        c.update(ctx_lo=_log_int(rng, 1, 64), ctx_hi=_log_int(rng, 64, 8192))
    elif op == "append":
        fp8 = rng.random() < 0.5
        c.update(R=_log_int(rng, 1, 256), gamma=_log_int(rng, 1, 60), ragged=rng.random() < 0.7,
                 Hkv=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 128]),
                 page=rng.choice([16, 32, 64, 128]), fp8=fp8, fused=rng.random() < 0.5)
        c.update(ctx_lo=_log_int(rng, 1, 64), ctx_hi=_log_int(rng, 64, 1024))
    elif op == "attn":
        tree = rng.random() < 0.5
        c.update(R=_log_int(rng, 1, 256), gamma=_log_int(rng, 1, 64) - 1, tree=tree,
                 ragged=rng.random() < 0.5)
        Hkv = rng.choice([1, 2, 4, 8])
        c.update(Hq=Hkv * rng.choice([1, 2, 4, 5, 8]), Hkv=Hkv, D=rng.choice([64, 128]),
                 page=rng.choice([16, 32, 64, 128]), fp8=rng.random() < 0.4,
                 fused=rng.random() < 0.5)
        lo = _log_int(rng, 1, 2048)
        c.update(ctx_lo=lo, ctx_hi=_log_int(rng, lo, 65536))
        # no dearer than the largest listed case, and the plain form's padded copies stay small
        while True:
            hi, rows = c["ctx_hi"] + c["gamma"] + 1, c["gamma"] + 1
            padded = c["R"] * hi * Hkv * c["D"] * 4
            scores = c["R"] * hi * c["Hq"] * rows * 4
            w = work(c)
            if padded <= 8e9 and scores <= 4e9 and w["bytes"] <= 1.5e9 and w["flops"] <= 1e11:
                break
            if c["ctx_hi"] > 2 * c["ctx_lo"]:
                c["ctx_hi"] = max(c["ctx_lo"], c["ctx_hi"] * 2 // 3)
            else:
                c["R"] = max(1, c["R"] * 2 // 3)
                c["ctx_lo"] = max(1, c["ctx_lo"] * 2 // 3)
                c["ctx_hi"] = max(c["ctx_lo"], c["ctx_hi"] * 2 // 3)
    elif op == "accept":
        c.update(R=_log_int(rng, 1, 1024), gamma=_log_int(rng, 1, 63), tree=rng.random() < 0.5,
                 ragged=rng.random() < 0.5, match=round(rng.uniform(0.3, 0.95), 3))
    else:
        c.update(R=_log_int(rng, 1, 256), gamma=_log_int(rng, 1, 31), tree=rng.random() < 0.8,
                 ragged=rng.random() < 0.5, Hkv=rng.choice([1, 2, 4, 8]),
                 D=rng.choice([64, 128]), page=rng.choice([16, 32, 64]), fp8=rng.random() < 0.4,
                 match=round(rng.uniform(0.3, 0.95), 3))
        c.update(ctx_lo=_log_int(rng, 1, 64), ctx_hi=_log_int(rng, 64, 512))
    return c


def _contexts(c):
    """The batch's context lengths: log-spaced over [ctx_lo, ctx_hi], in order."""
    R, lo, hi = c["R"], c["ctx_lo"], c["ctx_hi"]
    return [int(round(lo * (hi / lo) ** ((i + 0.5) / R))) for i in range(R)]


def _lengths(c):
    """Admitted drafts: every length 0..gamma in turn where ragged, else gamma."""
    return [i % (c["gamma"] + 1) if c["ragged"] else c["gamma"] for i in range(c["R"])]


def work(case):
    """Bytes and operations of one pass; the pairing of contexts with lengths is
    random, so the products of the two are taken at their means."""
    c, op = case, case["op"]
    R = c["R"]
    rows = sum(x + 1 for x in _lengths(c))
    if op == "accept":  # tokens, choices, parents; accepted, bonus, lengths, path
        return {"bytes": 4.0 * (rows * 2 + (rows if c["tree"] else 0) + R * (5 + c["gamma"])),
                "flops": 0}
    ctx = sum(_contexts(c))
    if op == "plan":  # lengths in; offsets, positions, slots, masks and new pages out
        pages = rows / c["page"]
        return {"bytes": 4.0 * R * 5 + (4.0 * rows if c["tree"] else 0) + rows * 20.0 + pages * 8,
                "flops": 0}
    vec = 2 * c["Hkv"] * c["D"]  # K and V values of one row
    size = 1 if c["fp8"] else 2
    if op == "append":
        return {"bytes": rows * (vec * (2.0 + size) + 8), "flops": 0}
    if op == "compact":  # the rows written once, and about a third of the nodes moved at most
        moved = R * min(c["gamma"], 1 / (1 - c["match"]))
        return {"bytes": rows * (vec * (2.0 + size) + 8) + 2.0 * moved * vec * size, "flops": 0}
    tokens = ctx + rows
    return {"bytes": tokens * vec * size + rows * c["Hq"] * (c["D"] * 4.0 + 4)
            + 4.0 * tokens / c["page"],
            "flops": 4.0 * c["Hq"] * c["D"] * rows * tokens / R}


# ----------------------------------------------------------------- inputs ----

def _parents(c, g):
    """Parent node of each draft node 1..gamma (node 0 is the anchor)."""
    R, G = c["R"], c["gamma"]
    j = torch.arange(1, G + 1, device="cuda")
    if not c.get("tree"):
        return (j - 1).expand(R, G).to(torch.int32).contiguous()
    back = (torch.rand((R, G), generator=g, device="cuda") ** 2 * j.clamp(max=6)).long()
    return (j - 1 - back).clamp(min=0).to(torch.int32).contiguous()


def _masks(parent, width):
    """Ancestor masks int64 [R, width] from parents [R, width - 1], by pointer doubling."""
    R = parent.shape[0]
    root = torch.zeros((R, 1), dtype=torch.long, device=parent.device)
    up = torch.cat([root, parent.long()], 1)
    bits = torch.ones_like(up) << torch.arange(width, device=parent.device)
    level = (bits, up)

    def double(level):
        b, u = level
        return b | b.gather(1, u), u.gather(1, u)

    # six doublings cover chains of 64 nodes; the root's parent is itself
    level = double(double(double(double(double(double(level))))))
    return level[0] | 1


def _depth(masks):
    """Ancestors of each node: the set bits of its mask, less itself."""
    return ((masks[..., None] >> torch.arange(64, device=masks.device)) & 1).sum(-1) - 1


def _rows(c, n):
    """Row offsets [R + 1] of `n` rows for each request, and each padded row's
    request, node and validity."""
    start = torch.cat([n.new_zeros(1), n.cumsum(0)])
    cap = c["R"] * (c["gamma"] + 1)
    row = torch.arange(cap, device="cuda")
    req = torch.searchsorted(start[1:].contiguous(), row, right=True).clamp(max=c["R"] - 1)
    return start, req, row - start[req], row < start[-1]


def _slots(c, start, req, node, valid, ctx, table):
    pos = ctx.long()[req] + node
    at = (pos // c["page"]).clamp(max=table.shape[1] - 1)
    slot = table[req, at].long() * c["page"] + pos % c["page"]
    return torch.where(valid, slot, -1)


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


def _new_rows(c, cap, g):
    """New K and V rows: views of one fused projection, or tensors of their own."""
    H, D = c["Hkv"], c["D"]
    if c.get("fused", True):
        both = torch.randn((cap, 2 * H, D), generator=g, device="cuda", dtype=torch.bfloat16)
        return both[:, :H], both[:, H:]
    return tuple(torch.randn((cap, H, D), generator=g, device="cuda", dtype=torch.bfloat16)
                 for _ in range(2))


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    R, G = c["R"], c["gamma"]
    s = dict(c=c)
    perm = lambda: torch.randperm(R, generator=g, device="cuda")  # noqa: E731
    length = torch.tensor(_lengths(c), dtype=torch.int32, device="cuda")[perm()].contiguous()
    s["len"] = length
    s["parent"] = _parents(c, g) if c.get("tree") else None
    start, req, node, valid = _rows(c, length.long() + 1)
    s["row_start"] = start.to(torch.int32)
    cap = R * (G + 1)
    if c["op"] in ("accept", "compact"):
        # each node's choice is one of its children's tokens with probability `match`
        parent = _parents(c, g) if s["parent"] is None else s["parent"]
        s["tokens"] = torch.randint(0, 32000, (R, max(G, 1)), generator=g, device="cuda",
                                    dtype=torch.int32)[:, :G].contiguous()
        choice = torch.randint(0, 32000, (R, G + 1), generator=g, device="cuda", dtype=torch.int32)
        pick = torch.rand((R, G), generator=g, device="cuda") < c["match"]
        at = torch.where(pick, parent.long(), G + 1)
        wide = torch.cat([choice, choice[:, :1]], 1)
        # the last picked child is the node's choice: node order decides, not the scatter's
        child = torch.full((R, G + 2), -1, dtype=torch.long, device="cuda")
        child.scatter_reduce_(1, at, torch.arange(G, device="cuda").expand(R, G), "amax")
        got = child.gather(1, torch.arange(G + 2, device="cuda").expand(R, G + 2))
        if G:
            wide = torch.where(got >= 0, s["tokens"].gather(1, got.clamp(min=0)), wide)
        s["choice"] = torch.where(valid, wide[req, node.clamp(max=G)], -1).to(torch.int32)
    if c["op"] == "accept":
        s["ctx"] = torch.randint(0, 8192, (R,), generator=g, device="cuda", dtype=torch.int32)
        return s
    s["ctx"] = torch.tensor(_contexts(c), dtype=torch.int32, device="cuda")[perm()].contiguous()
    ps = c["page"]
    s["max_pages"] = -(-(c["ctx_hi"] + G + 2) // ps)
    need = -(-(s["ctx"].long() + length.long() + 1) // ps)
    n_pages = sum(-(-(x + G + 2) // ps) for x in _contexts(c)) + 8
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    if c["op"] == "plan":
        # pages held for the committed tokens; the rest are on the free stack
        held = -(-s["ctx"].long() // ps)
        s["held"], s["n_pages"] = held.to(torch.int32), n_pages
        table, used = _deal(order, held, s["max_pages"])
        s["table"], s["free"] = table, torch.cat([order[used:], order[:used]]).contiguous()
        s["n_free"] = torch.tensor([n_pages - used], dtype=torch.int32, device="cuda")
        if c["leave"]:  # every 16th request has finished: its pages go back
            s["ctx"] = torch.where(perm() % 16 == 0, -1, s["ctx"]).to(torch.int32)
        return s
    s["table"], _ = _deal(order, need, s["max_pages"])
    s.update(_cache(c, n_pages, g))
    s["slot"] = _slots(c, start, req, node, valid, s["ctx"], s["table"])
    if c["op"] in ("append", "compact"):
        s["k"], s["v"] = _new_rows(c, cap, g)
    if c["op"] == "compact":
        s["ctx_before"] = s["ctx"]
        s["accepted"], _, s["path"], _ = plain_accept(s)
    if c["op"] == "attn":
        masks = _masks(_parents(c, g) if s["parent"] is None else s["parent"], G + 1)
        s["anc"] = torch.where(valid, masks[req, node.clamp(max=G)], 0)
        wide = c["Hq"] + (2 * c["Hkv"] if c["fused"] else 0)
        s["q"] = (2.0 * torch.randn((cap, wide, c["D"]), generator=g, device="cuda",
                                    dtype=torch.bfloat16))[:, :c["Hq"]]
        s["out"] = torch.zeros((cap, c["Hq"], c["D"]), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.zeros((cap, c["Hq"]), dtype=torch.float32, device="cuda")
    return s


def _deal(order, pages, max_pages):
    """Block table of the first pages of `order`, and how many it took."""
    first = pages.cumsum(0) - pages
    col = torch.arange(max_pages, device="cuda")
    at = (first[:, None] + col).clamp(max=order.numel() - 1)
    table = torch.where(col < pages[:, None], order[at], -1)
    return table.to(torch.int32).contiguous(), int(pages.sum())


# ------------------------------------------------------------ plain forms ----

def plain_plan(s):
    c = s["c"]
    R, G, ps = c["R"], c["gamma"], c["page"]
    ctx, held, gone = s["ctx"].long(), s["held"].long(), s["ctx"] < 0
    rows = torch.where(gone, 0, s["len"].long() + 1)
    start, req, node, valid = _rows(c, rows)
    col = torch.arange(s["max_pages"], device="cuda")
    # finished requests' pages onto the stack, in request order
    back = torch.where(gone, held, 0)
    at = s["n_free"].long() + (back.cumsum(0) - back)[:, None] + col
    returned = col < back[:, None]
    free = torch.cat([s["free"], s["free"][:1]])
    free[torch.where(returned, at, s["n_pages"])] = torch.where(returned, s["table"], 0)
    top = s["n_free"].long() + back.sum()
    # the new rows' pages off its top
    need = torch.where(gone, 0, -(-(ctx + rows) // ps) - held).clamp(min=0)
    last = need.cumsum(0)
    k = (last - need - held)[:, None] + col
    fresh = (col >= held[:, None]) & (col < (held + need)[:, None])
    table = torch.where(fresh, free[(top - 1 - k).clamp(0, s["n_pages"] - 1)], s["table"])
    if c["tree"]:
        masks = _masks(s["parent"], G + 1)
    else:
        masks = ((2 << torch.arange(G + 1, device="cuda")) - 1).expand(R, G + 1)
    own_mask = masks[req, node.clamp(max=G)]
    position = ctx[req] + _depth(own_mask)
    return dict(row_start=start.to(torch.int32),
                position=torch.where(valid, position, -1).to(torch.int32),
                slot=_slots(c, start, req, node, valid, s["ctx"], table),
                anc=torch.where(valid, own_mask, 0), table=table,
                held=(held - back + need).to(torch.int32), free=free[:-1],
                n_free=(top - last[-1]).to(torch.int32))


def plain_append(s):
    c = s["c"]
    keep = s["slot"] >= 0
    # padded rows write where the last row of their batch does, with that row's values
    final = keep.sum() - 1
    row = torch.where(keep, torch.arange(keep.numel(), device="cuda"), final)
    slot = s["slot"][row]
    page, at = slot // c["page"], slot % c["page"]
    for_k = _stored(s["k"], s.get("k_scale"))[row]
    for_v = _stored(s["v"], s.get("v_scale"))[row]
    raw = (lambda t: t.view(torch.uint8)) if c["fp8"] else (lambda t: t)
    raw(s["kc"])[page, at] = raw(for_k)
    raw(s["vc"])[page, at] = raw(for_v)
    return s["kc"], s["vc"]


def _stored(x, scale):
    if scale is None:
        return x
    return (x.float() / scale[:, None]).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)


def plain_attn(s):
    c = s["c"]
    R, W, H, D = c["R"], c["gamma"] + 1, c["Hkv"], c["D"]
    rep = c["Hq"] // H
    start = s["row_start"].long()
    nodes = start[1:] - start[:-1]
    row = start[:-1, None] + torch.arange(W, device="cuda")
    row_ok = torch.arange(W, device="cuda") < nodes[:, None]
    row = torch.where(row_ok, row, 0)
    L = s["max_pages"] * c["page"]
    pos = torch.arange(L, device="cuda")
    inside = pos < (s["ctx"].long() + nodes)[:, None]
    table = s["table"].long().clamp(min=0)

    def gathered(x, scale):  # [R, H, L, D] in f32, zero past the request's end
        raw = x.view(torch.uint8)[table].view(x.dtype) if c["fp8"] else x[table]
        y = raw.view(R, L, H, D).float()
        if scale is not None:
            y = y * scale[:, None]
        return torch.where(inside[:, :, None, None], y, 0.0).permute(0, 2, 1, 3)

    q = s["q"][row].float().view(R, W, H, rep, D).permute(0, 2, 1, 3, 4).reshape(R, H, W * rep, D)
    score = (q @ gathered(s["kc"], s.get("k_scale")).transpose(2, 3)) * (1 / math.sqrt(D))
    bit = (pos - s["ctx"].long()[:, None])                                   # [R, L]
    drafted = ((s["anc"][row][:, :, None] >> bit.clamp(0, 63)[:, None]) & 1).bool()
    seen = ((bit < 0)[:, None] | (drafted & (bit < 64)[:, None])) & inside[:, None]  # [R, W, L]
    seen = seen[:, None, :, None].expand(R, 1, W, rep, L).reshape(R, 1, W * rep, L)
    score = score.masked_fill_(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = p @ gathered(s["vc"], s.get("v_scale")) / torch.where(total == 0, 1.0, total)
    lse = (top + torch.log(total)).squeeze(-1)
    back = lambda t: t.view(R, H, W, rep, -1).permute(0, 2, 1, 3, 4).reshape(R * W, H * rep, -1)  # noqa: E731
    to = torch.where(row_ok, row, R * W).reshape(-1)  # padded rows go to a row of their own
    out = torch.zeros((R * W + 1, c["Hq"], D), dtype=torch.bfloat16, device="cuda")
    out[to] = back(o).to(torch.bfloat16)
    lse_out = torch.zeros((R * W + 1, c["Hq"]), device="cuda")
    lse_out[to] = back(lse).squeeze(-1)
    return out[:-1], lse_out[:-1]


def plain_accept(s):
    c = s["c"]
    R, G = c["R"], c["gamma"]
    start = s["row_start"].long()
    nodes = (start[1:] - start[:-1])[:, None]
    node = torch.arange(1, G + 1, device="cuda")
    parent = (node - 1).expand(R, G) if s["parent"] is None else s["parent"].long()
    last = s["choice"].numel() - 1
    wanted = s["choice"][(start[:-1, None] + parent).clamp(max=last)]
    hit = (s["tokens"] == wanted) & (node < nodes)
    # of several matching children of one node the lowest is taken
    same = (parent[:, :, None] == parent[:, None, :]) & hit[:, None, :] & (node[None, :] < node[:, None])
    hit = hit & ~same.any(-1)
    ok = torch.cat([hit.new_ones((R, 1)), hit], 1)
    bits = (ok.long() << torch.arange(G + 1, device="cuda")).sum(1, keepdim=True)
    masks = _masks(parent, G + 1)
    on = ((masks & ~bits) == 0)[:, 1:]                   # every node up to the root matched
    count = on.sum(1)
    end = torch.where(on, node, 0).amax(1) if G else count
    order = torch.where(on, on.long().cumsum(1) - 1, G)
    path = torch.full((R, G + 1), -1, dtype=torch.int32, device="cuda")
    path.scatter_(1, order, torch.where(on, node, -1).to(torch.int32))
    bonus = s["choice"][(start[:-1] + end).clamp(max=last)]
    return (count.to(torch.int32), bonus, path[:, :G].contiguous(),
            (s["ctx"].long() + 1 + count).to(torch.int32))


def plain_compact(s):
    c = s["c"]
    plain_append(s)
    ps, G = c["page"], c["gamma"]
    j = torch.arange(1, G + 1, device="cuda")
    moves = j <= s["accepted"][:, None]
    ctx = s["ctx"].long()[:, None]
    src = ctx + torch.where(moves, s["path"].long(), 0)
    dst = ctx + torch.where(moves, j, 0)   # a move that is none puts the anchor's row on itself
    req = torch.arange(c["R"], device="cuda")[:, None]
    slot = lambda p: (s["table"][req, p // ps].long(), p % ps)  # noqa: E731
    raw = (lambda t: t.view(torch.uint8)) if c["fp8"] else (lambda t: t)
    kc, vc = raw(s["kc"]), raw(s["vc"])
    k, v = kc[slot(src)], vc[slot(src)]
    kc[slot(dst)] = k
    vc[slot(dst)] = v
    return s["kc"], s["vc"]


PLAIN = dict(plan=plain_plan, append=plain_append, attn=plain_attn, accept=plain_accept,
             compact=plain_compact)


# -------------------------------------------------- the framework's calls ----

def own_plan(s):
    import speculative_decoding_draft_02_gb300 as dsp
    c = s["c"]
    R, cap = c["R"], c["R"] * (c["gamma"] + 1)
    if "o" not in s:
        new = lambda shape, t: torch.empty(shape, dtype=t, device="cuda")  # noqa: E731
        s["o"] = dict(row_start=new(R + 1, torch.int32), position=new(cap, torch.int32),
                      slot=new(cap, torch.int64), anc=new(cap, torch.int64), table=s["table"],
                      free=s["free"], held=new(R, torch.int32), n_free=new(1, torch.int32))
    o = s["o"]
    dsp.dspark_kv_plan(s["ctx"], s["len"], 1, s["parent"], c["page"], s["held"], s["n_free"],
                       s["free"], s["table"], o["held"], o["n_free"], o["row_start"],
                       o["position"], o["slot"], o["anc"])
    return o


def _own_cache(s):
    import speculative_decoding_draft_02_gb300 as dsp
    if "cache" not in s:
        s["cache"] = dsp.KVCache(s["kc"], s["vc"], s.get("k_scale"), s.get("v_scale"))
    return dsp, s["cache"]


def own_append(s):
    dsp, cache = _own_cache(s)
    dsp.dspark_kv_append(cache, s["k"], s["v"], s["slot"])
    return s["kc"], s["vc"]


def own_attn(s):
    dsp, cache = _own_cache(s)
    c = s["c"]
    if "ws" not in s:
        s["ws"] = dsp.workspace(dsp.dspark_tree_attention_workspace_bytes(
            cache, c["R"], c["Hq"], c["gamma"] + 1))
    dsp.dspark_tree_attention(cache, s["q"], s["ctx"], s["row_start"], s["anc"], s["table"],
                              c["gamma"] + 1, 1 / math.sqrt(c["D"]), s["out"], s["lse"], s["ws"])
    return s["out"], s["lse"]


def own_accept(s):
    import speculative_decoding_draft_02_gb300 as dsp
    c = s["c"]
    if "o" not in s:
        new = lambda *n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
        s["o"] = (new(c["R"]), new(c["R"]), new(c["R"], c["gamma"]), new(c["R"]))
    dsp.dspark_tree_accept(s["row_start"], s["parent"], s["tokens"], s["choice"], s["ctx"], *s["o"])
    return s["o"]


def own_compact(s):
    dsp, cache = _own_cache(s)
    dsp.dspark_kv_append(cache, s["k"], s["v"], s["slot"])
    dsp.dspark_kv_compact(cache, s["ctx"], s["accepted"], s["path"], s["table"])
    return s["kc"], s["vc"]


OWN = dict(plan=own_plan, append=own_append, attn=own_attn, accept=own_accept,
           compact=own_compact)


def run(state):
    return (OWN if own else PLAIN)[state["c"]["op"]](state)


# ------------------------------------------------------------ in 64 bits ----

def exact(case, seed):
    c = case
    if c["op"] in ("plan", "accept"):
        return None  # whole numbers
    s = prepare(case, seed)
    R, ps = c["R"], c["page"]
    start, ctx, table = s["row_start"].tolist(), s["ctx"].tolist(), s["table"].cpu()
    if c["op"] == "attn":
        return _exact_attn(c, s, start, ctx, table)
    slot = s["slot"].tolist()
    kept = torch.tensor([x for x in slot if x >= 0], device="cuda")
    caches = []
    for x in ("k", "v"):
        cache = s[x + "c"].double().view(-1, c["Hkv"], c["D"])
        new = s[x][:len(kept)].double()
        if c["fp8"]:
            new = (new / s[x + "_scale"].double()[:, None]).clamp(-FP8_MAX, FP8_MAX)
            new = new.float().to(torch.float8_e4m3fn).double() if c["op"] == "compact" else new
        cache[kept] = new
        caches.append(cache)
    if c["op"] == "compact":
        accepted, path = s["accepted"].tolist(), s["path"].tolist()
        place = lambda r, p: int(table[r, p // ps]) * ps + p % ps  # noqa: E731
        src = [place(r, ctx[r] + path[r][j]) for r in range(R) for j in range(accepted[r])]
        dst = [place(r, ctx[r] + 1 + j) for r in range(R) for j in range(accepted[r])]
        if src:
            src, dst = (torch.tensor(x, device="cuda") for x in (src, dst))
            for cache in caches:
                cache[dst] = cache[src]
    return tuple(cache.view(s["kc"].shape) for cache in caches)


def _exact_attn(c, s, start, ctx, table):
    H, D, Hq, ps = c["Hkv"], c["D"], c["Hq"], c["page"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    for r in range(c["R"]):
        n = start[r + 1] - start[r]
        pages = table[r, :-(-(ctx[r] + n) // ps)].long().cuda()
        kv = []
        for x in ("k", "v"):
            y = torch.cat([s[x + "c"][int(p)][None].double() for p in pages]) if c["fp8"] \
                else s[x + "c"][pages].double()
            y = y.reshape(-1, H, D)[:ctx[r] + n]
            kv.append(y * s[x + "_scale"].double()[:, None] if c["fp8"] else y)
        k, v = (y.repeat_interleave(Hq // H, 1) for y in kv)
        q = s["q"][start[r]:start[r + 1]].double()
        z = torch.einsum("nhd,thd->hnt", q, k) / math.sqrt(D)
        hide = torch.zeros((n, ctx[r] + n), dtype=torch.bool)
        for i, word in enumerate(s["anc"][start[r]:start[r + 1]].tolist()):
            for j in range(n):
                hide[i, ctx[r] + j] = not (word >> j) & 1
        z = z.masked_fill(hide.cuda(), -math.inf)
        lse[start[r]:start[r + 1]] = torch.logsumexp(z, -1).t()
        out[start[r]:start[r + 1]] = torch.einsum("hnt,thd->nhd", torch.softmax(z, -1), v)
    return out, lse
