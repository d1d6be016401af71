"""The paged KV cache of a verification round in plain loops and float64.

Covers what the target model's pass over a round's rows needs of its cache:
rows, pages, slots and ancestor masks (kv_plan), the rows written (kv_append),
attention of a drafted tree over the cache (tree_attention), the path of the
tree that the target confirms (tree_accept) and its K and V moved together
(kv_compact).  Written from the definitions, one request and one token at a
time; shares no code with the CUDA path.
"""
from __future__ import annotations

import math

import numpy as np


def e4m3_values() -> np.ndarray:
    """The 256 values of an 8-bit float of 4 exponent (bias 7) and 3 mantissa bits
    without infinities: codes 0x7f and 0xff are NaN."""
    out = np.empty(256)
    for code in range(256):
        sign, exp, man = -1.0 if code & 0x80 else 1.0, (code >> 3) & 15, code & 7
        if exp == 15 and man == 7:
            out[code] = np.nan
        elif exp == 0:
            out[code] = sign * man * 2.0 ** -9
        else:
            out[code] = sign * (1 + man / 8) * 2.0 ** (exp - 7)
    return out


def e4m3_round(x: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value, halves to the even code, saturating at +-448; NaN stays."""
    pos = e4m3_values()[:127]                      # ascending, code by code
    a = np.minimum(np.abs(np.asarray(x, dtype=np.float64)), 448.0)
    hi = np.clip(np.searchsorted(pos, np.nan_to_num(a)), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - pos[lo], pos[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return np.where(np.isnan(x), np.nan, np.copysign(pos[code], x))


def ancestors(parent, n: int):
    """Sets {node and its ancestors} of nodes 0..n-1; parent[j-1] is node j's."""
    sets = []
    for j in range(n):
        sets.append({j} | (sets[parent[j - 1]] if j else set()))
    return sets


def kv_plan(ctx, length, extra, parent, page_size, held, n_free, free_pages, block_table, n_rows):
    """Returns a dict of every output; inputs are left alone.  parent None: chains."""
    free_pages, table = np.array(free_pages), np.array(block_table)
    held, top = np.array(held), int(n_free)
    R = len(ctx)
    n = [0 if ctx[r] < 0 else int(length[r]) + extra for r in range(R)]
    for r in range(R):
        if ctx[r] < 0:
            for b in range(held[r]):
                free_pages[top] = table[r, b]
                top += 1
            held[r] = 0
    starved = False
    for r in range(R):
        need = 0 if ctx[r] < 0 else max(0, -(-(int(ctx[r]) + n[r]) // page_size) - int(held[r]))
        if need and (starved or need > top):
            starved = True
            table[r, held[r]:held[r] + need] = -1
            continue
        for _ in range(need):
            top -= 1
            table[r, held[r]] = free_pages[top]
            held[r] += 1
    row_start = np.concatenate([[0], np.cumsum(n)]).astype(np.int64)
    position, slot = np.full(n_rows, -1), np.full(n_rows, -1)
    anc = np.zeros(n_rows, dtype=np.uint64)
    for r in range(R):
        chain = list(range(n[r]))
        sets = ancestors(chain if parent is None else parent[r], n[r]) if n[r] <= 64 else None
        for i in range(n[r]):
            row, pos = row_start[r] + i, int(ctx[r]) + i
            if row >= n_rows:
                continue
            position[row] = ctx[r] + (len(sets[i]) - 1 if sets else i)
            if pos // page_size < held[r]:
                slot[row] = table[r, pos // page_size] * page_size + pos % page_size
            if sets:
                anc[row] = sum(1 << j for j in sets[i])
    return dict(row_start=np.minimum(row_start, n_rows), position=position, slot=slot, anc=anc,
                held=held, n_free=top, free_pages=free_pages, block_table=table)


def kv_append(cache, new, slot, scale=None):
    """cache [n_pages, page_size, heads, dim] after the rows `new` [rows, heads, dim];
    scale [heads]: an e4m3 cache, held as the values its codes stand for (before the
    scale)."""
    out = np.array(cache, dtype=np.float64)
    ps = out.shape[1]
    for row, s in enumerate(slot):
        if 0 <= s < out.shape[0] * ps:
            x = np.asarray(new[row], dtype=np.float64)
            if scale is not None:
                # the quotient is an f32 one
                x = e4m3_round((x.astype(np.float32)
                                / np.asarray(scale, np.float32)[:, None]).astype(np.float64))
            out[s // ps, s % ps] = x
    return out


def tree_attention(q, k, v, ctx, row_start, anc, block_table, scale, k_scale=None, v_scale=None):
    """(out [rows, heads_q, dim], lse [rows, heads_q]) in f64; k, v [n_pages, page_size,
    heads, dim]; anc None: chains.  Padding rows are 0."""
    rows, heads_q, dim = q.shape
    ps, heads = k.shape[1], k.shape[2]
    out, lse = np.zeros(q.shape), np.zeros((rows, heads_q))
    for r in range(len(ctx)):
        row0, n = int(row_start[r]), int(row_start[r + 1] - row_start[r])
        for i in range(n):
            word = (2 << i) - 1 if anc is None else int(anc[row0 + i])
            seen = list(range(int(ctx[r]))) + [int(ctx[r]) + j for j in range(n) if word >> j & 1]
            page = [int(block_table[r, p // ps]) for p in seen]
            at = [p % ps for p in seen]
            for h in range(heads_q):
                g = h // (heads_q // heads)
                if not seen:
                    lse[row0 + i, h] = -math.inf
                    continue
                kk = k[page, at, g].astype(np.float64) * (1.0 if k_scale is None else k_scale[g])
                vv = v[page, at, g].astype(np.float64) * (1.0 if v_scale is None else v_scale[g])
                s = scale * (kk @ q[row0 + i, h].astype(np.float64))
                top = s.max()
                w = np.exp(s - top)
                out[row0 + i, h] = w @ vv / w.sum()
                lse[row0 + i, h] = top + math.log(w.sum())
    return out, lse


def tree_accept(row_start, parent, tokens, choice, ctx):
    """(accepted, bonus, paths as lists, ctx_out); parent None: chains."""
    accepted, bonus, paths, ctx_out = [], [], [], []
    for r in range(len(ctx)):
        row0, n = int(row_start[r]), int(row_start[r + 1] - row_start[r])
        cur, path = 0, []
        while n:
            nxt = [j for j in range(1, n)
                   if (j - 1 if parent is None else parent[r][j - 1]) == cur
                   and tokens[r][j - 1] == choice[row0 + cur]]
            if not nxt:
                break
            cur = nxt[0]
            path.append(cur)
        accepted.append(len(path))
        bonus.append(int(choice[row0 + cur]) if n else -1)
        paths.append(path)
        ctx_out.append(int(ctx[r]) + (1 + len(path) if n else 0))
    return accepted, bonus, paths, ctx_out


def kv_compact(cache, ctx, paths, block_table):
    """cache [n_pages, page_size, heads, dim] with every request's path moved together."""
    src, out = np.array(cache), np.array(cache)
    ps = out.shape[1]
    for r, path in enumerate(paths):
        for j, node in enumerate(path):
            a, b = int(ctx[r]) + node, int(ctx[r]) + 1 + j
            out[block_table[r, b // ps], b % ps] = src[block_table[r, a // ps], a % ps]
    return out
