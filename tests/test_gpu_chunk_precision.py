"""With how many bits the chunk attention's weights meet V: one bf16 number beside a bf16
cache, f16 beside an 8-bit one, and a sum that takes them unrounded.

Scores are exact (K and q small whole numbers, the scale a power of two), all rows of a KV
head have the same q, and V is chosen so that sum_p w_p V_p nearly vanishes: an output is then
its rounding, 2^-8 |out| with |out| tiny, and what the weights lost.  That is known value by
value: with r(w) the weight over the first tile's largest, rounded as promised, an output is
off by D = sum_p (r(w_p) - w_p) V_p / sum_p w_p, or by less where fewer bits are lost.  The
bound is |D| and, with A = sum_p w_p |V_p| / sum_p w_p,
  2^-21 A           ex2's own error, 2^-22, in a weight and in the sum
  6 ln2 S 2^-24 A   the exponent's roundings, S the largest |score| in log2 units
  n 2^-24 A         f32 additions of n tokens
  one step of a weight that these could carry over the middle between two roundings
Items of so few tokens are not cut, so that every row has one reference.  Weights of 8 bits
where 11 are promised, or of 6 where 8 are, pass the bound: shown in f64, without the kernel.
"""
import math

import numpy as np
import pytest
import torch

from test_gpu_cache import dsp, host, _lib  # noqa: F401
from test_gpu_cache_precision import LOG2E, cancelling_values
from test_gpu_chunk import run

pytestmark = pytest.mark.gpu

TYPES = pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])


def rounded(w, bits):
    """To so many bits, ties to even: no weight here is below 2^-20 of the largest."""
    m, e = np.frexp(w)
    return np.ldexp(np.rint(m * 2.0 ** bits), e - bits)


@TYPES
@pytest.mark.parametrize("R", [1, 80])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group,nodes", [(1, 70), (4, 33), (8, 64), (5, 60), (16, 20), (64, 3)])
def test_bits_of_a_weight(group, nodes, dim, R, fp8):
    rng = np.random.default_rng(100 * group + nodes)
    ctx, ps, heads, scale = 300, 16, 2, 0.25
    n = ctx + nodes
    pages, (bits, too_few) = -(-n // ps), (11, 8) if fp8 else (8, 6)
    k = rng.integers(-1, 2, (pages * ps, heads, dim)).astype(np.float64)
    q1 = rng.integers(-1, 2, (heads, dim)).astype(np.float64)
    v = np.zeros((pages * ps, heads, dim))
    want, bound, fewer = (np.zeros((nodes, heads, dim)) for _ in range(3))
    for h in range(heads):
        s = scale * (k[:n, h] @ q1[h])
        w = np.exp(s - s[:128].max())   # over the first tile's largest, as every row has them
        assert w.min() > 2.0 ** -20 * w.max()
        v[:ctx, h] = cancelling_values(rng, w[:ctx], dim, fp8)   # and zeros in the rows' own
        sums = np.cumsum(w)[ctx:, None]
        a, av = w[:ctx], v[:ctx, h]
        slip = 2.0 ** -21 + 6 * math.log(2) * scale * np.abs(k[:n, h] @ q1[h]).max() * LOG2E * 2.0 ** -24
        step = np.abs(rounded(a * (1 + slip), bits) - rounded(a * (1 - slip), bits))
        lost = np.abs((rounded(a, bits) - a) @ av)
        want[:, h] = (a @ av) / sums
        bound[:, h] = (lost + step @ np.abs(av) + (slip + n * 2.0 ** -24) * (a @ np.abs(av))) / sums
        fewer[:, h] = np.abs(rounded(a, too_few) @ av) / sums
    dtype = torch.float8_e4m3fn if fp8 else torch.bfloat16
    shaped = lambda x: torch.tensor(x.reshape(pages, ps, heads, dim)).to(dtype).cuda()  # noqa: E731
    ones = [torch.ones(heads, device="cuda") for _ in range(2)] if fp8 else []
    rows = R * nodes
    q = torch.tensor(np.repeat(q1, group, 0)[None].repeat(rows, 0)).to(torch.bfloat16).cuda()
    c = dict(cache=dsp.KVCache(shaped(k), shaped(v), *ones), ctx=np.full(R, ctx), ns=[nodes] * R, q=q,
             scale=scale, row_start=np.arange(R + 1) * nodes, table=np.tile(np.arange(pages), (R, 1)))
    out, lse = run(c)
    got = np.float64(host(out)).reshape(R, nodes, heads, group, dim)
    tol = 2.0 ** -8 * np.abs(want) + bound
    err = np.abs(got - want[None, :, :, None])
    assert (err <= tol[None, :, :, None]).all(), np.max(err / tol[None, :, :, None])
    assert (fewer > tol + np.abs(want)).mean() > 0.5
