"""A prompt's way into the paged cache in plain loops and float64.

Norm and rotation of heads (rope_append), attention of chunks of new rows
(chunk_attention), and pages with several holders: continuations (kv_fork), pages
given back (kv_release), the pages in use moved to the lowest numbers (kv_squeeze)
and the copies that these leave (kv_copy).  Written from the definitions, one
request and one value at a time; shares no code with the CUDA path.
"""
from __future__ import annotations

import math

import numpy as np

from .cache import e4m3_round


def norm_rotate(x, weight, eps, inv_freq, pairs, position):
    """One head [dim] at one position."""
    x = np.array(x, dtype=np.float64)
    if weight is not None:
        x = x / math.sqrt(np.mean(x * x) + eps) * weight
    half = len(inv_freq)
    for i, f in enumerate(inv_freq):
        a, b = (2 * i, 2 * i + 1) if pairs else (i, i + half)
        c, s = math.cos(position * f), math.sin(position * f)
        x[a], x[b] = x[a] * c - x[b] * s, x[b] * c + x[a] * s
    return x


def rope_append(q, k, v, position, slot, inv_freq, pairs, q_weight, k_weight, eps, q_out, k_cache,
                v_cache, k_scale=None, v_scale=None):
    """(q_out, k_cache, v_cache) after the rows; the first two unrounded where they are written,
    and an e4m3 cache's keys before the rounding to it; caches [n_pages, page_size, heads, dim]."""
    q_out, k_cache, v_cache = (np.array(t, dtype=np.float64) for t in (q_out, k_cache, v_cache))
    ps = k_cache.shape[1]
    for m, p in enumerate(position):
        if p < 0:
            continue
        for h in range(q.shape[1]):
            q_out[m, h] = norm_rotate(q[m, h], q_weight, eps, inv_freq, pairs, int(p))
        s = int(slot[m])
        if 0 <= s < k_cache.shape[0] * ps:
            for h in range(k.shape[1]):
                y = norm_rotate(k[m, h], k_weight, eps, inv_freq, pairs, int(p))
                k_cache[s // ps, s % ps, h] = y if k_scale is None else y / k_scale[h]
                x = np.asarray(v[m, h], dtype=np.float64)
                v_cache[s // ps, s % ps, h] = x if v_scale is None else e4m3_round(
                    (x.astype(np.float32) / np.float32(v_scale[h])).astype(np.float64))
    return q_out, k_cache, v_cache


def chunk_attention(q, k, v, ctx, row_start, block_table, scale, k_scale=None, v_scale=None):
    """(out [rows, heads_q, dim], lse [rows, heads_q], size): `size` is the weighted mean of
    |V|, what roundings of the weights are relative to.  Padding rows are 0."""
    rows, heads_q, dim = q.shape
    ps, heads = k.shape[1], k.shape[2]
    out, size, lse = np.zeros(q.shape), np.zeros(q.shape), np.zeros((rows, heads_q))
    for r in range(len(ctx)):
        row0, n = int(row_start[r]), int(row_start[r + 1] - row_start[r])
        if n == 0:
            continue
        pos = np.arange(min(int(ctx[r]) + n, block_table.shape[1] * ps))
        page = block_table[r][pos // ps]
        for h in range(heads_q):
            g = h // (heads_q // heads)
            kk = k[page, pos % ps, g].astype(np.float64) * (1.0 if k_scale is None else k_scale[g])
            vv = v[page, pos % ps, g].astype(np.float64) * (1.0 if v_scale is None else v_scale[g])
            for i in range(n):
                e = min(int(ctx[r]) + i + 1, len(pos))
                s = scale * (kk[:e] @ q[row0 + i, h].astype(np.float64))
                w = np.exp(s - s.max())
                out[row0 + i, h] = w @ vv[:e] / w.sum()
                size[row0 + i, h] = w @ np.abs(vv[:e]) / w.sum()
                lse[row0 + i, h] = s.max() + math.log(w.sum())
    return out, lse, size


def kv_fork(source, target, page_size, ctx, held, n_free, free_pages, block_table, refs):
    """A dict of everything after the forks."""
    ctx, held, table, refs = (np.array(t) for t in (ctx, held, block_table, refs))
    before, held_before, R, top = ctx.copy(), held.copy(), len(ctx), int(n_free)
    copies, starved, seen, bad = [], False, set(), 0
    for s, d in zip(source, target):
        copies.append((-1, -1, 0))
        if s < 0:
            continue
        first = d not in seen
        seen.add(int(d))
        if not (s < R and 0 <= d < R and before[s] >= 0 and before[d] < 0 and held_before[d] == 0
                and first and -(-before[s] // page_size) <= held_before[s]):
            bad += 1
            continue
        full, tail = divmod(int(before[s]), page_size)
        if tail and (starved or top == 0):
            starved = True
            continue
        for j in range(full):
            table[d, j] = table[s, j]
            refs[table[s, j]] += 1
        if tail:
            top -= 1
            table[d, full] = free_pages[top]
            copies[-1] = (int(table[s, full]), int(free_pages[top]), tail)
        ctx[d], held[d] = before[s], full + (tail > 0)
    return dict(ctx=ctx, held=held, n_free=top, block_table=table, refs=refs,
                copies=np.array(copies).reshape(-1, 3), starved=starved, bad=bad)


def kv_release(ctx, held, n_free, free_pages, block_table, refs):
    """A dict of everything after the pages went back."""
    held, free, refs = (np.array(t) for t in (held, free_pages, refs))
    top = int(n_free)
    left = [(r, j) for r in range(len(ctx)) if ctx[r] < 0 for j in range(held[r])]
    holds = {}
    for r, j in left:
        holds.setdefault(int(block_table[r, j]), []).append((r, j))
    for r, j in left:
        page = int(block_table[r, j])
        if len(holds[page]) == refs[page] + 1 and holds[page][-1] == (r, j):
            free[top] = page
            top += 1
    for page, by in holds.items():
        refs[page] = max(refs[page] - len(by), 0)
    held[np.array(ctx) < 0] = 0
    return dict(held=held, n_free=top, free_pages=free, refs=refs)


def kv_squeeze(held, n_free, free_pages, block_table, refs):
    """A dict of everything after the pages in use have the lowest numbers."""
    n, n_free = len(free_pages), int(n_free)
    free = set(int(p) for p in free_pages[:n_free])
    used = n - n_free
    goes = [p for p in range(used, n) if p not in free]
    takes = sorted(p for p in free if p < used)
    new_page = np.array([-1 if p in free else p for p in range(n)])
    new_page[goes] = takes
    table, out = np.array(block_table), np.zeros(n, dtype=np.int64)
    for r in range(len(held)):
        for j in range(held[r]):
            table[r, j] = new_page[table[r, j]]
    for p in range(n):
        if new_page[p] >= 0:
            out[new_page[p]] = refs[p]
    stack = np.array(free_pages)
    stack[:n_free] = [n - 1 - i for i in range(n_free)]
    fill = [-1] * (n // 2 - len(goes))
    return dict(free_pages=stack, block_table=table, refs=out, new_page=new_page,
                move_from=np.array(goes + fill), move_to=np.array(takes + fill), n_moves=len(goes))


def kv_copy(cache, copy_from, copy_to, tokens=None):
    """cache [n_pages, page_size, heads, dim] after the copies."""
    out = np.array(cache)
    for i, (a, b) in enumerate(zip(copy_from, copy_to)):
        if a >= 0:
            n = out.shape[1] if tokens is None else tokens[i]
            out[b, :n] = cache[a, :n]
    return out
