"""The paged-cache operators where they turn from one way to another: every width of
the attention's row tiles, scores that climb past any reference, scores without a
finite value, more nodes allowed than present, captured graphs, pages that come and
go, and the 8-bit rounding of every bf16 value.

The attention is held to the float64 oracle with the tolerances of test_gpu_cache.
Where scores grow past 100 they are whole numbers here, exact in f32, and what is
added comes from their way into an exponential: the scale, log2(e) and the
difference round once each, at most 5 * 2^-24 |score| in a weight's exponent, which
an output's numerator and denominator have both: 10 * 2^-24 max|score| of A.  Beside
an 8-bit cache weights are f16, which has a least step, 2^-24: half of it for each
token, beside a largest weight of at least 2^6, is 2^-31 sum_p |v_p| (it shows where
the only token with weight has a zero in V).
"""
import math

import numpy as np
import pytest
import torch

from oracle import cache as oc
from test_gpu_cache import (U, attention_case, check_attention, dsp, host, i32, make_cache,
                            run_attention, _lib)  # noqa: F401

pytestmark = pytest.mark.gpu

TYPES = pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])


@TYPES
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group,nodes", [(1, 1), (16, 1), (1, 17), (8, 4), (3, 11), (8, 6), (1, 49),
                                         (16, 4), (5, 13), (2, 64), (43, 3), (64, 2), (33, 7),
                                         (49, 2)])
def test_row_tiles(group, nodes, dim, fp8):
    ctx = [0, 127, 401, 640]
    ns = [nodes, max(nodes - 1, 0), nodes, 1]
    c = attention_case(ctx, ns, 2 * group, 2, dim, 16, fp8=fp8, seed=group * 100 + nodes)
    out, lse = run_attention(c)
    check_attention(c, out, lse)
    again, lse2 = run_attention(c)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@TYPES
@pytest.mark.parametrize("shape", ["up", "down", "spike", "late", "saw"])
@pytest.mark.parametrize("group,nodes", [(2, 3), (4, 10), (4, 30)])
def test_scores_that_climb(group, nodes, shape, fp8):
    # K's first column takes 16 levels along the context, q's first column 64, 0, -64:
    # the scores of neighbouring rows climb, stay or fall by 240
    n_ctx, dim = 700, 64
    c = attention_case([n_ctx, 50], [nodes, 2], 2 * group, 2, dim, 16, fp8=fp8, seed=nodes)
    p = np.arange(n_ctx)
    level = dict(up=p * 16 // n_ctx, down=15 - p * 16 // n_ctx, spike=15 * (p == 333),
                 late=15 * (p >= 690), saw=(p * 5) % 16)[shape]
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    cache = c["cache"]
    k = torch.randint(-1, 2, cache.k.shape, generator=g, device="cuda").float()
    table = c["table"][0]
    k[torch.tensor(table[p // 16], device="cuda"), torch.tensor(p % 16, device="cuda"), :, 0] = \
        torch.tensor(level, device="cuda").float()[:, None]
    cache.k.copy_(k.to(cache.k.dtype))
    q = torch.randint(-1, 2, c["q"].shape, generator=g, device="cuda").float()
    q[:, :, 0] = 64.0 * (torch.arange(q.shape[0] * q.shape[1], device="cuda") % 3 - 1).view(
        q.shape[:2])
    c["q"] = q.to(torch.bfloat16)
    c["scale"] = 0.25
    out, lse = run_attention(c)
    qd, kd, vd = (np.float64(host(t)) for t in (c["q"], cache.k, cache.v))
    ks, vs = (None if s is None else np.float64(host(s)) for s in (cache.k_scale, cache.v_scale))
    args = (c["ctx"], c["row_start"], c["anc"], c["table"], c["scale"])
    want, want_lse = oc.tree_attention(qd, kd, vd, *args, ks, vs)
    size, _ = oc.tree_attention(qd, kd, np.abs(vd), *args, ks, vs)
    total = int(c["row_start"][-1])
    most = 0.25 * (64 * 15 + dim) * (1.25 if fp8 else 1.0)
    got, want, size = np.float64(host(out))[:total], want[:total], size[:total]
    tol = U * np.abs(want) + (U + 2e-4 + 10 * 2.0 ** -24 * most) * size
    if fp8:
        tol += 2.0 ** -31 * (n_ctx + nodes) * np.nanmax(np.abs(vd)) * vs.max()
    err = np.abs(got - want)
    assert (err <= tol).all(), np.max(err / tol)
    bound = 5 * 2.0 ** -24 * most + np.spacing(np.float32(most)) + 1e-5
    assert (np.abs(np.float64(host(lse))[:total] - want_lse[:total]) <= bound).all()


@pytest.mark.parametrize("group,nodes", [(2, 3), (4, 10), (4, 30)])
@pytest.mark.parametrize("tokens", [[0], list(range(128)), list(range(300)), [200], [128, 300]])
def test_scores_of_minus_infinity(tokens, group, nodes):
    # those tokens have no weight in the rows whose q is above zero there, and make
    # NaN of the others
    c = attention_case([301], [nodes], 2 * group, 2, 64, 16, seed=3)
    q = c["q"].clone()
    q[:, :, 9] = 1.0
    q[:, 0, 9] = -1.0
    c["q"] = q
    for p in tokens:
        c["cache"].k[c["table"][0, p // 16], p % 16, :, 9] = -math.inf
    out, lse = run_attention(c)
    with np.errstate(invalid="ignore"):
        rest = slice(1, None)
        qd, kd, vd = (np.float64(host(t)) for t in (c["q"], c["cache"].k, c["cache"].v))
        args = (c["ctx"], c["row_start"], c["anc"], c["table"], c["scale"])
        want, want_lse = oc.tree_attention(qd, kd, vd, *args)
        size, _ = oc.tree_attention(qd, kd, np.abs(vd), *args)
    assert np.isnan(want[:nodes, 0]).all() and np.isnan(host(out)[:nodes, 0]).all()
    got, want, size = (np.float64(x)[:nodes, rest] for x in (host(out), want, size))
    assert np.isfinite(want).all()
    assert (np.abs(got - want) <= U * np.abs(want) + (U + 2e-4) * size + 1e-30).all()
    np.testing.assert_allclose(host(lse)[:nodes, rest], want_lse[:nodes, rest], atol=1e-3, rtol=0)


@TYPES
def test_nan_in_the_context_reaches_every_row(fp8):
    for which in ("k", "v"):
        c = attention_case([150], [5], 8, 2, 64, 16, fp8=fp8, seed=8)
        t = getattr(c["cache"], which)
        row = t[c["table"][0, 0], 0].float()
        row[0, 3] = math.nan       # the first token, first head
        t[c["table"][0, 0], 0] = row.to(t.dtype)
        out, lse = run_attention(c)
        bad = np.isnan(host(out)[:5])
        if which == "k":
            assert bad[:, :4].all()
        else:
            assert bad[:, :4, 3].all() and not bad[:, :4, 4:].any()
        assert not bad[:, 4:].any()


@TYPES
def test_more_nodes_allowed_than_present(fp8):
    c = attention_case([90, 0, 300], [3, 1, 6], 8, 2, 128, 32, fp8=fp8, seed=12)
    for most in (6, 7, 33, 64):
        out, lse = run_attention(c, max_nodes=most)
        check_attention(c, out, lse)


@TYPES
def test_captured_round(fp8):
    # append and attention in a graph, replayed over new rows, against direct calls
    c = attention_case([140, 20], [4, 4], 8, 2, 128, 16, fp8=fp8, seed=14, poison=False)
    cache, rows = c["cache"], 8
    slot = torch.tensor([int(c["table"][r, p // 16]) * 16 + p % 16 for r, x in enumerate((140, 20))
                         for p in range(x, x + 4)], device="cuda")
    new = torch.zeros((2, rows, 2, 128), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((rows, 8, 128), dtype=torch.bfloat16, device="cuda")
    ws = dsp.workspace(dsp.dspark_tree_attention_workspace_bytes(cache, 2, 8, 4))
    anc = torch.tensor(c["anc"].view(np.int64)[:rows], device="cuda")
    ctx, row_start, table = i32(c["ctx"]), i32(c["row_start"]), i32(c["table"])
    out = torch.zeros_like(q)

    def step():
        dsp.dspark_kv_append(cache, new[0], new[1], slot)
        dsp.dspark_tree_attention(cache, q, ctx, row_start, anc, table, 4, 0.1, out, None, ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        new.copy_(torch.randn(new.shape, generator=g, device="cuda"))
        q.copy_(torch.randn(q.shape, generator=g, device="cuda"))
        out.zero_()
        graph.replay()
        got = out.clone()
        out.zero_()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, out) and (got != 0).any()


def test_page_pool_gives_pages_back():
    pool = dsp.PagePool(3, 10, 16, 100, 64)
    pool.ctx.copy_(i32([0, 0, -1]))
    pool.plan(i32([33, 16, 0]), extra=0)
    assert host(pool.n_free)[0] == 6 and host(pool.held).tolist() == [3, 1, 0]
    pool.commit(i32([33, 16, 0]))
    assert host(pool.ctx).tolist() == [33, 16, -1]
    pool.plan(i32([5, 5, 5]))                    # rounds of 6 rows; the third place is free
    assert host(pool.held).tolist() == [3, 2, 0] and host(pool.n_free)[0] == 5
    assert host(pool.row_start).tolist() == [0, 6, 12, 12]
    pool.ctx[0] = -1                             # the first leaves
    pool.plan(i32([5, 5, 5]))
    assert host(pool.held).tolist() == [0, 2, 0] and host(pool.n_free)[0] == 8
    held = set(host(pool.block_table)[1, :2].tolist())
    free = set(host(pool.free_pages)[:8].tolist())
    assert held | free == set(range(10)) and not held & free


def test_append_rounds_every_bf16_as_its_quotient():
    # all bf16 patterns over scales whose reciprocals are exact, inexact, too small and
    # too large for the short way
    bits = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16)
    x = bits.view(torch.bfloat16).view(64, 8, 128)
    scales = [1.0, 0.25, 3.0, 1 / 3, 0.7, 1e-35, 3e33, 1.0859375, 2.0 ** -90, 5e-29, 0.013, 448.0,
              1 / 448, 1.1, 57.0, 2.0 ** -130]
    slot = torch.arange(64, device="cuda")
    xs = host(x)
    with np.errstate(all="ignore"):
        for shift in range(16):
            cache = make_cache(4, 16, 8, 128, True, seed=shift)
            ks, vs = (torch.tensor((scales[shift:] + scales[:shift])[i:i + 8], device="cuda")
                      for i in (0, 8))
            cache = dsp.KVCache(cache.k, cache.v, ks, vs)
            dsp.dspark_kv_append(cache, x, x, slot)
            for got, s in ((cache.k, ks), (cache.v, vs)):
                want = oc.e4m3_round((xs / host(s)[:, None]).astype(np.float64))
                np.testing.assert_array_equal(host(got).reshape(64, 8, 128), want)
