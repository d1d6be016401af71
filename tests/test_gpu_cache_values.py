"""Infinities in committed values, which meet a weight's two parts."""
import math

import numpy as np
import pytest
import torch

from test_gpu_cache import attention_case, host, run_attention, _lib  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group,nodes,ctx", [(1, 1, 40), (4, 3, 150), (4, 10, 301), (16, 3, 700),
                                             (4, 30, 700), (2, 3, 9000)])
@pytest.mark.parametrize("dim", [64, 128])
def test_infinities_in_committed_values(group, nodes, ctx, dim):
    # a bf16 weight is two numbers, the second of either sign or zero: an infinite value
    # must meet it once.  Column 3 has +inf, 5 -inf, 7 both: inf, -inf, NaN in every row.
    c = attention_case([ctx, 9], [nodes, 1], 2 * group, 2, dim, 16, seed=ctx)
    clean, clean_lse = run_attention(c)
    v = c["cache"].v
    for col, places in ((3, [0, ctx // 3]), (5, [ctx // 2]), (7, [1, ctx - 1])):
        for i, p in enumerate(places):
            value = math.inf if col == 3 or (col == 7 and i) else -math.inf
            v[c["table"][0, p // 16], p % 16, :, col] = value
    out, lse = run_attention(c)
    assert torch.equal(lse, clean_lse)
    got = host(out)[:nodes]
    assert (got[:, :, 3] == math.inf).all() and (got[:, :, 5] == -math.inf).all()
    assert np.isnan(got[:, :, 7]).all()
    rest = [i for i in range(dim) if i not in (3, 5, 7)]
    assert torch.equal(out[:nodes][:, :, rest], clean[:nodes][:, :, rest])
    assert torch.equal(out[nodes:], clean[nodes:])
