"""With how many bits the attention's weights meet V, and Q the keys: what the public
header promises, at inputs where nothing else can hide it.

Weights.  K and q are small whole numbers and the scale a power of two, so scores are
exact; all rows of a KV head have the same q, and V is chosen (in f64, value by value)
so that sum_p w_p V_p nearly vanishes.  An output then is its rounding, 2^-8 |out|
at most with |out| tiny, plus what the weights lost: with A = sum_p w_p |V_p| / sum_p w_p
  2^-16 A   two bf16 numbers a weight (half a step of 8 bits, 2^-8 at most, twice), or
  2^-11 A   f16 (half a step of 11 bits, down to 2^-20 of the largest), and half of its
            least step a token beside a largest weight of 2^6 or more: 2^-31 sum_p |V_p|
  2^-21 A   ex2's own error, 2^-22, in a weight and in the factors that join pieces
  6 ln2 S 2^-24 A   the exponent's roundings, S the largest |score| in log2 units: the
            score times log2(e) (its constant and the sum, each 2^-24 of 2 S at most),
            and the references of two pieces and their difference
  n 2^-24 A   f32 additions of n tokens, 16 and what is summed so far a step, each of the
            17 cut at 2^-24 of the largest at worst
The same rows with weights of fewer bits than promised (one bf16 number, or four bits
beside an 8-bit cache) are off by more than that: shown in f64, without the kernel.

Q beside an 8-bit cache is f16 under one power of two a tile, its 8 bits whole down to
2^-28 of the tile's largest value.
"""
import math

import numpy as np
import pytest
import torch

from oracle import cache as oc
from test_gpu_cache import (attention_case, check_attention, dsp, host, run_attention,
                            _lib)  # noqa: F401

pytestmark = pytest.mark.gpu

TYPES = pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
LOG2E = 1.4426950408889634


def bf16(x):
    return np.float64(torch.tensor(x, dtype=torch.float64).to(torch.bfloat16).double().numpy())


def cancelling_values(rng, w, dim, fp8):
    """V [tokens, dim] of the cache's type with sum_p w_p V_p near zero."""
    fit = oc.e4m3_round if fp8 else bf16
    v = fit(rng.normal(size=(len(w), dim)))
    rest = w @ v
    for p in np.argsort(-w)[:40]:        # from the heaviest token on, ever finer
        new = fit(np.clip(v[p] - rest / w[p], -6, 6))
        rest = rest + w[p] * (new - v[p])
        v[p] = new
    return v


def fewer_bits(w, fp8):
    """Weights over their largest, rounded to what the kernel must not use."""
    return oc.e4m3_round(w * 256 / w.max()) if fp8 else bf16(w / w.max())


@TYPES
@pytest.mark.parametrize("R", [1, 80])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group,nodes", [(1, 1), (4, 2), (8, 4), (8, 6), (16, 4), (4, 30)])
def test_bits_of_a_weight(group, nodes, dim, R, fp8):
    rng = np.random.default_rng(10 * group + nodes)
    ctx, ps, heads, scale = 300, 16, 2, 0.25
    pages = -(-(ctx + nodes) // ps)
    k = rng.integers(-1, 2, (pages * ps, heads, dim)).astype(np.float64)
    q1 = rng.integers(-1, 2, (heads, dim)).astype(np.float64)
    v = np.zeros((pages * ps, heads, dim))
    top = 0.0
    for h in range(heads):
        s = scale * (k[:ctx, h] @ q1[h])
        top = max(top, scale * np.abs(k[:, h] @ q1[h]).max() * LOG2E)
        w = np.exp(s - s.max())
        v[:ctx, h] = cancelling_values(rng, w, dim, fp8)
    # every row of every request reads the same pages: the nodes' V are zeros
    dtype = torch.float8_e4m3fn if fp8 else torch.bfloat16
    shaped = lambda x: torch.tensor(x.reshape(pages, ps, heads, dim)).to(dtype).cuda()  # noqa: E731
    ones = [torch.ones(heads, device="cuda") for _ in range(2)] if fp8 else []
    cache = dsp.KVCache(shaped(k), shaped(v), *ones)
    rows = R * nodes
    q = torch.tensor(np.repeat(q1, group, 0)[None].repeat(rows, 0)).to(torch.bfloat16).cuda()
    c = dict(cache=cache, ctx=np.full(R, ctx), ns=[nodes] * R, anc=None, q=q, scale=scale,
             row_start=np.arange(R + 1) * nodes, table=np.tile(np.arange(pages), (R, 1)))
    out, lse = run_attention(c)
    one = (host(q)[:nodes].astype(np.float64), k.reshape(pages, ps, heads, dim))
    vv = v.reshape(pages, ps, heads, dim)
    args = (c["ctx"][:1], c["row_start"][:2], None, c["table"][:1], scale)
    want, _ = oc.tree_attention(*one, vv, *args)
    size, _ = oc.tree_attention(*one, np.abs(vv), *args)
    n = ctx + nodes
    part = 2.0 ** -11 if fp8 else 2.0 ** -16
    tol = 2.0 ** -8 * np.abs(want) + (part + 2.0 ** -21 + 6 * math.log(2) * top * 2.0 ** -24
                              + n * 2.0 ** -24) * size
    if fp8:
        tol += 2.0 ** -31 * np.abs(vv).sum((0, 1)).repeat(group, 0)[None]
    got = np.float64(host(out)).reshape(R, nodes, heads * group, dim)
    err = np.abs(got - want)
    assert (err <= tol).all(), np.max(err / tol)
    # the planted mistake, in f64: weights of too few bits pass the bound
    for h in range(heads):
        s = scale * (k[:ctx, h] @ q1[h])
        w = np.exp(s - s.max())
        off = np.abs(fewer_bits(w, fp8) @ v[:ctx, h] / fewer_bits(w, fp8).sum())
        assert (off > tol[0, h * group]).mean() > 0.5


@pytest.mark.parametrize("power", [-27, 0, 12])
@pytest.mark.parametrize("group,nodes", [(2, 3), (4, 10), (16, 4)])
def test_rows_of_very_different_size_share_a_tile(group, nodes, power):
    # one query head is 2^27 times as large as the others (in a column where K is zero):
    # beside an 8-bit cache its neighbours keep their bits
    c = attention_case([200, 31], [nodes, 2], 2 * group, 2, 64, 16, fp8=True, seed=nodes)
    k = c["cache"].k
    f = k.float()
    f[..., 11] = torch.where(torch.isnan(f[..., 11]), f[..., 11], 0.0)
    k.copy_(f.to(k.dtype))
    q = c["q"].float()
    q[:, :, 11] = 0.0
    q[:, 0] = 0.0
    q[0, 0, 11] = q.abs().max() * 2.0 ** 27
    c["q"] = (q * 2.0 ** power).to(torch.bfloat16)
    c["scale"] *= 2.0 ** -power
    out, lse = run_attention(c)
    check_attention(c, out, lse)
