"""Attention of chunks of new rows against the float64 oracle, through the C-ABI.

Tolerances, per element, with A = sum_p w_p |v_p| / sum_p w_p from the oracle:
  out: 2^-8 |out| for its own rounding (half a step of bf16 at most), 2^-8 A for the
       weights' rounding to bf16, and for f32 arithmetic e A with
       e = 2 d + 2^-20, d = dim 2^-23 max_p scale sum_i |q_i k_i|
       (a score's dim additions and products, in any order, shift its weight and, by as
       much, the sum; exponentials are off by 2^-22, sums of n weights by far less than
       n 2^-24 as 128 at a time are added)
  lse: d + 1e-5
"""
import math

import numpy as np
import pytest
import torch

from oracle import prompt as op
from test_gpu_cache import attention_case, dsp, host, i32, _lib  # noqa: F401

pytestmark = pytest.mark.gpu

TYPES = pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
U = 2.0 ** -8


def case(ctx, ns, heads_q, heads, dim, ps, fp8=False, **kw):
    return attention_case(ctx, ns, heads_q, heads, dim, ps, fp8, tree=False, **kw)


def run(c, max_rows=None, stream=None, ws=None, want_lse=True):
    cache, q = c["cache"], c["q"]
    rows, heads_q, dim = q.shape
    out = torch.full((rows, heads_q + 1, dim), -77.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((rows, heads_q), -77.0, device="cuda") if want_lse else None
    max_rows = max_rows or max(max(c["ns"]), 1)
    if ws is None:
        ws = dsp.workspace(dsp.dspark_chunk_attention_workspace_bytes(cache, len(c["ctx"]), heads_q,
                                                                      max_rows))
        ws.fill_(255)  # contents on entry are ignored: NaN patterns
    args = (cache, q, i32(c["ctx"]), i32(c["row_start"]), i32(c["table"]), max_rows, c["scale"],
            out[:, :heads_q], lse, ws)
    torch.cuda.synchronize()
    dsp.dspark_chunk_attention(*args, stream=stream)
    torch.cuda.synchronize()
    assert (out[:, heads_q] == -77).all()
    return out[:, :heads_q], lse


def check(c, out, lse):
    cache = c["cache"]
    q, k, v = (np.float64(host(t)) for t in (c["q"], cache.k, cache.v))
    ks, vs = (None if s is None else np.float64(host(s)) for s in (cache.k_scale, cache.v_scale))
    want, want_lse, size = op.chunk_attention(q, k, v, c["ctx"], c["row_start"], c["table"], c["scale"],
                                              ks, vs)
    total = int(c["row_start"][-1])
    got, got_lse = np.float64(host(out)), np.float64(host(lse))
    assert (got[total:] == -77).all() and (got_lse[total:] == -77).all()
    top = np.nanmax(np.abs(k)) * (1 if ks is None else ks.max())
    d = (q.shape[2] * 2.0 ** -23 * c["scale"] * np.abs(q).sum(-1) * top)[:total]
    err = np.abs(got[:total] - want[:total])
    tol = U * np.abs(want[:total]) + (U + 2 * d[..., None] + 2.0 ** -20) * size[:total]
    assert (err <= tol).all(), np.nanmax(err / tol)
    off = np.abs(got_lse - want_lse)[:total]
    assert (off <= d + 1e-5).all(), np.max(off / (d + 1e-5))


CASES = {
    # ctx, rows, heads_q, heads, dim, page
    "one_row": ([0], [1], 1, 1, 64, 16),
    "one_row_far": ([1000], [1], 8, 2, 128, 16),
    "a_tile_less_one": ([0], [127], 2, 2, 128, 32),
    "a_tile": ([0], [128], 4, 1, 64, 64),
    "a_tile_and_one": ([1], [129], 3, 3, 128, 128),
    "two_tiles_and_one": ([0], [257], 1, 1, 128, 16),
    "group_of_five": ([33, 0], [77, 130], 10, 2, 128, 16),
    "group_of_seven": ([10], [200], 7, 1, 64, 32),
    "group_of_64": ([100], [70], 64, 1, 128, 16),
    "ragged": ([0, 700, 5, 130, 64, 0, 255], [70, 1, 300, 0, 65, 129, 2], 8, 2, 128, 16),
    "mixed_64": ([300, 31, 0, 512], [3, 100, 190, 66], 8, 4, 64, 256),
    "empty_requests": ([50, 0, 9, 3], [0, 0, 90, 0], 4, 2, 64, 16),
    "long_context": ([5000], [80], 4, 2, 128, 64),
    "wide_batch": ([17 * i for i in range(40)], [65 + i % 3 for i in range(40)], 2, 1, 64, 32),
}


@TYPES
@pytest.mark.parametrize("name", CASES)
def test_matches_oracle(name, fp8):
    c = case(*CASES[name], fp8=fp8, seed=len(name))
    out, lse = run(c)
    check(c, out, lse)
    again, lse2 = run(c)   # the same bits from call to call
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@TYPES
@pytest.mark.parametrize("order", ["head", "padded"])
def test_strides(order, fp8):
    c = case([40, 0], [90, 150], 6, 2, 128, 32, fp8=fp8, order=order, seed=3)
    check(c, *run(c))


@TYPES
def test_the_bound_on_rows_is_only_a_bound(fp8):
    # few rows by themselves, and with a bound that says nothing: both within tolerance
    c = case([0, 200, 40], [5, 64, 33], 8, 2, 128, 16, fp8=fp8, seed=8)
    check(c, *run(c))
    check(c, *run(c, max_rows=100000))
    check(c, *run(c, max_rows=2 ** 31 - 1))


@pytest.mark.parametrize("max_rows", [70, 130])
def test_rows_past_the_bound_are_not_computed(max_rows):
    c = case([3, 0], [200, 75], 4, 2, 64, 16, seed=4)
    want, _ = run(c)
    out, lse = run(c, max_rows=max_rows)
    assert dsp.dspark_device_status() == 6
    np.testing.assert_allclose(host(out[:max_rows]), host(want[:max_rows]), rtol=2 ** -7, atol=2e-2)
    assert (out[max_rows:200] == -77).all() and (lse[max_rows:200] == -77).all()
    done = min(75, max_rows)
    np.testing.assert_allclose(host(out[200:200 + done]), host(want[200:200 + done]), rtol=2 ** -7,
                               atol=2e-2)


@TYPES
@pytest.mark.parametrize("dim", [64, 128])
def test_values_of_later_rows_do_not_reach_earlier_ones(dim, fp8):
    # infinities and NaN in V of a chunk's rows: seen from their row on, by nobody before
    n, ctx, ps = 300, 45, 16
    c = case([ctx, 7], [n, 70], 4, 2, dim, ps, fp8=fp8, seed=dim)
    clean, clean_lse = run(c)
    v, table = c["cache"].v, c["table"]
    marks = {2: math.nan, 90: math.nan if fp8 else math.inf, 200: math.nan if fp8 else -math.inf,
             299: math.nan}
    raw = v.float()
    for node, value in marks.items():
        p = ctx + node
        raw[table[0, p // ps], p % ps, 1, 5 + node % 3] = value
    v.copy_(raw.to(v.dtype))
    out, lse = run(c)
    total = n + 70
    assert torch.equal(lse[:total], clean_lse[:total])
    got, want = host(out), host(clean)
    group = 2
    for col in range(dim):
        first = min([node for node in marks if 5 + node % 3 == col], default=n)
        # the KV head 1's query heads
        assert np.array_equal(got[:first, group:, col], want[:first, group:, col]), col
        assert not np.isfinite(got[first:n, group:, col]).any()
    assert np.array_equal(got[:total, :group], want[:total, :group])
    assert np.array_equal(got[n:total], want[n:total])


def test_infinities_in_committed_values():
    n, ctx, ps = 140, 500, 32
    c = case([ctx], [n], 4, 2, 128, ps, seed=2)
    clean, clean_lse = run(c)
    v, table = c["cache"].v, c["table"]
    for p, col, value in ((3, 1, math.inf), (400, 2, -math.inf), (7, 3, math.inf), (490, 3, -math.inf)):
        v[table[0, p // ps], p % ps, :, col] = value
    out, lse = run(c)
    got, want = host(out)[:n], host(clean)[:n]
    assert torch.equal(lse[:n], clean_lse[:n])
    assert (got[..., 1] == math.inf).all() and (got[..., 2] == -math.inf).all()
    assert np.isnan(got[..., 3]).all()
    rest = [i for i in range(128) if i not in (1, 2, 3)]
    assert np.array_equal(got[..., rest], want[..., rest])


@TYPES
def test_scores_that_climb_and_fall(fp8):
    # references raised late, by a lot, and never lowered; constant scores
    c = case([0, 600], [400, 150], 2, 1, 64, 16, fp8=fp8, seed=5, q_std=1.0)
    k, table = c["cache"].k, c["table"]
    raw = k.float()
    for r, total in ((0, 400), (1, 750)):
        for p in range(total):
            raw[table[r, p // 16], p % 16, 0, 0] = (p if r == 0 else total - p) / 8.0
    k.copy_(raw.to(k.dtype))
    c["q"][:, :, 0] = 20.0
    check(c, *run(c))
    c["q"].zero_()
    check(c, *run(c))


def test_negative_scale():
    c = case([30], [200], 2, 1, 64, 16, seed=16)
    c["scale"] = -c["scale"]
    out, lse = run(c)
    c["scale"], c["q"] = -c["scale"], -c["q"]   # the same scores
    want, want_lse = run(c)
    assert torch.equal(out[:200], want[:200]) and torch.equal(lse[:200], want_lse[:200])
    check(c, want, want_lse)


def test_large_finite_values():
    c = case([100], [100], 2, 1, 128, 16, seed=6)
    c["cache"].v.mul_(2.0 ** 60)
    check(c, *run(c))


@TYPES
def test_queries_and_keys_that_are_no_numbers(fp8):
    n, ctx = 150, 20
    c = case([ctx], [n], 2, 1, 64, 16, fp8=fp8, seed=7)
    clean, clean_lse = run(c)
    c["q"][70, 1, 3] = math.nan
    p = ctx + 100                       # a key that rows from 100 on see
    raw = c["cache"].k.float()
    raw[c["table"][0, p // 16], p % 16, 0, 9] = math.nan
    c["cache"].k.copy_(raw.to(c["cache"].k.dtype))
    out, lse = run(c)
    got, want = host(out), host(clean)
    assert np.isnan(got[100:n]).all() and np.isnan(got[70, 1]).all()
    keep = np.ones((n, 2), dtype=bool)
    keep[70, 1] = keep[100:] = False
    assert np.array_equal(got[:n][keep], want[:n][keep])
    assert np.array_equal(host(lse)[:n][keep], host(clean_lse)[:n][keep])
    assert np.isnan(host(lse)[100:n]).all()


@TYPES
def test_bad_pages_read_as_zeros(fp8):
    c = case([100], [100], 4, 2, 64, 16, fp8=fp8, seed=9)
    for bad in (-1, 10 ** 6):
        c["table"][0, 3] = bad
        out, lse = run(c)
        assert dsp.dspark_device_status() == 9
        assert np.isfinite(host(out[:100])).all()
    # as a page of zeros would
    zero = c["cache"].n_pages - 1
    free = [p for p in range(c["cache"].n_pages) if p not in set(c["table"].ravel())]
    zero = free[0]
    for t in (c["cache"].k, c["cache"].v):
        raw = t.float()
        raw[zero] = 0
        t.copy_(raw.to(t.dtype))
    c["table"][0, 3] = zero
    want, want_lse = run(c)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_a_request_longer_than_its_table():
    c = case([100], [200], 2, 1, 64, 16, seed=10)
    cut = dict(c, table=np.ascontiguousarray(c["table"][:, :10]))
    out, lse = run(cut)
    assert dsp.dspark_device_status() == 6
    check(cut, out, lse)


def test_places_that_were_left():
    c = case([0, 60], [80, 90], 2, 1, 64, 16, seed=11)
    c["row_start"] = np.array([0, 0, 80, 170])
    c["ctx"] = np.array([-1, 0, 60])
    c["table"] = np.concatenate([np.full((1, c["table"].shape[1]), -1), c["table"]])
    c["ns"] = [0, 80, 90]
    check(c, *run(c))


def test_on_another_stream_and_without_lse():
    c = case([0, 60], [80, 190], 4, 2, 128, 16, seed=12)
    want, _ = run(c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, _ = run(c, stream=s, want_lse=False)
    assert torch.equal(got, want)


def test_in_a_graph_beside_calls():
    c = case([0, 900], [300, 190], 4, 2, 128, 16, seed=13)
    want, want_lse = run(c)
    cache, q, R = c["cache"], c["q"], 2
    need = dsp.dspark_chunk_attention_workspace_bytes(cache, R, 4, 300)
    ws = [dsp.workspace(need) for _ in range(2)]
    args = (cache, q, i32(c["ctx"]), i32(c["row_start"]), i32(c["table"]), 300, c["scale"])
    outs = [torch.zeros(want.shape, dtype=want.dtype, device="cuda") for _ in range(2)]
    lses = [torch.zeros_like(want_lse) for _ in range(2)]
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        dsp.dspark_chunk_attention(*args, outs[0], lses[0], ws[0])
    for _ in range(5):
        with torch.cuda.stream(s):
            g.replay()
        dsp.dspark_chunk_attention(*args, outs[1], lses[1], ws[1])
    torch.cuda.synchronize()
    total = int(c["row_start"][-1])
    for o, l in zip(outs, lses):
        assert torch.equal(o[:total], want[:total]) and torch.equal(l[:total], want_lse[:total])


def test_offsets_past_32_bits():
    # pages spread over 9 GB of a cache's elements
    ps, heads, dim = 16, 1, 64
    big = torch.zeros((2 ** 32 + 2 ** 27,), dtype=torch.bfloat16, device="cuda")
    n_pages = 40
    stride = (big.numel() // (n_pages + 1)) // 64 * 64
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    views = [big.as_strided((n_pages, ps, heads, dim), (stride, heads * dim, dim, 1), off)
             for off in (0, 1 << 20)]
    for v in views:
        v.copy_(torch.randn(v.shape, generator=g, device="cuda"))
    cache = dsp.KVCache(*views)
    c = case([200], [300], 2, 1, 64, ps, seed=14, poison=False)
    c["cache"], c["table"] = cache, np.random.default_rng(3).permutation(n_pages)[None]
    check(c, *run(c))


def test_a_prompt_in_chunks_is_the_prompt_at_once():
    n, heads_q, heads, dim, ps = 700, 8, 2, 128, 32
    c = case([0], [n], heads_q, heads, dim, ps, seed=15)
    whole, whole_lse = run(c)
    for cuts in ([0, 1, 66, 300, 700], [0, 350, 351, 700]):
        for a, b in zip(cuts, cuts[1:]):
            part = dict(c, ctx=np.array([a]), ns=[b - a], row_start=np.array([0, b - a]), q=c["q"][a:b + 3])
            out, lse = run(part)
            # both within the tolerance of the same numbers
            np.testing.assert_allclose(host(lse)[:b - a], host(whole_lse)[a:b], rtol=1e-5, atol=1e-4)
            off = np.abs(host(out)[:b - a] - host(whole)[a:b])
            assert off.max() <= 4 * U * np.abs(host(whole)[:n]).max()
