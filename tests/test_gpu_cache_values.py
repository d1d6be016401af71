"""Infinities in committed values, which meet a weight's two parts; and strides of
dimensions of one element, which mean nothing."""
import math

import numpy as np
import pytest
import torch

from test_gpu_cache import attention_case, dsp, host, i32, run_attention, _lib  # noqa: F401

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


@pytest.mark.parametrize("order", ["row", "head"])
def test_one_row_of_a_large_buffer(order):
    # a single row's stride is never stepped by, whatever it is in the buffer around it
    heads_q, dim, n = 32, 128, 6000
    c = attention_case([77], [1], heads_q, 8, dim, 16, seed=5)
    want, _ = run_attention(c)
    args = (i32(c["ctx"]), i32(c["row_start"]), None, i32(c["table"]), 1, c["scale"])
    q = c["q"][:1].contiguous()
    shape = (n, heads_q, dim) if order == "row" else (heads_q, n, dim)
    big = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    view = big[17:18] if order == "row" else big[:, 17:18].transpose(0, 1)
    ws = dsp.workspace(dsp.dspark_tree_attention_workspace_bytes(c["cache"], 1, heads_q, 1))
    dsp.dspark_tree_attention(c["cache"], q, *args, view, None, ws)
    assert torch.equal(view, want[:1])
    big.zero_()
    # and as a view that carries a stride of its own for that dimension
    odd = big.as_strided((1, heads_q, dim), (1 << 30, view.stride(1), 1), view.storage_offset())
    dsp.dspark_tree_attention(c["cache"], q, *args, odd, None, ws)
    assert torch.equal(view, want[:1])


@pytest.mark.parametrize("ns", [[1], [5, 0, 3]], ids=["one_row", "rows"])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_head_major_queries_and_outputs(ns, fp8):
    heads_q, dim, rows = 8, 64, sum(ns)
    c = attention_case([77, 3, 300][:len(ns)], ns, heads_q, 2, dim, 16, fp8=fp8, seed=6)
    want, want_lse = run_attention(c)
    q, out = (torch.zeros((heads_q, 40 + rows, dim), dtype=torch.bfloat16, device="cuda")
              for _ in range(2))
    q[:, 9:9 + rows] = c["q"][:rows].transpose(0, 1)
    anc = torch.tensor(c["anc"].view(np.int64)[:rows], device="cuda")
    lse = torch.zeros((rows, heads_q), device="cuda")
    ws = dsp.workspace(dsp.dspark_tree_attention_workspace_bytes(c["cache"], len(ns), heads_q, 5))
    dsp.dspark_tree_attention(c["cache"], q[:, 9:9 + rows].transpose(0, 1), i32(c["ctx"]),
                              i32(c["row_start"]), anc, i32(c["table"]), 5, c["scale"],
                              out[:, 3:3 + rows].transpose(0, 1), lse, ws)
    np.testing.assert_allclose(host(out[:, 3:3 + rows].transpose(0, 1)), host(want[:rows]),
                               rtol=2.0 ** -7, atol=1e-3)
    np.testing.assert_allclose(host(lse), host(want_lse[:rows]), rtol=1e-4, atol=1e-4)
    assert (out[:, :3] == 0).all() and (out[:, 3 + rows:] == 0).all()
