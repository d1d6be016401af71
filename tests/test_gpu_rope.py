"""Norm, rotation and append of a prompt's rows against the float64 oracle.

Tolerances, from the arithmetic.  A result is a cos t - b sin t of f32 values a, b: the
norm's sum of at most 128 squares is off by at most 64 * 2^-24 after its root, its
reciprocal and the two products by 4 * 2^-24 more, the angle by pi * 2^-25 (the fraction
of a turn rounded to f32) and its sine and cosine by 2^-23, the last sum by 2^-24: below
2^-17 (|a| + |b|) in all, and |a| + |b| is at most twice the head's largest result (the
rotation keeps a^2 + b^2).  On top comes one rounding: 2^-8 of the value in bf16, 2^-4 of
it in e4m3 (2^-10 below 2^-6).  Values are appended as they are: equal.
"""
import math

import numpy as np
import pytest
import torch

from oracle import prompt as op
from test_gpu_cache import dsp, host, i32, make_cache, _lib  # noqa: F401

pytestmark = pytest.mark.gpu

F32 = 2.0 ** -16  # 2^-17 (|a| + |b|) in parts of the head's largest result


def inv_freq(rot, base=1e4):
    return base ** (-np.arange(rot // 2) * 2.0 / max(rot, 1))


def rows_case(rows, heads_q, heads, dim, seed, fused=True, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    both = (std * torch.randn((rows, heads_q + 2 * heads, dim), generator=g, device="cuda")).to(
        torch.bfloat16)
    parts = both[:, :heads_q], both[:, heads_q:heads_q + heads], both[:, heads_q + heads:]
    weights = [(1 + 0.3 * torch.randn((dim,), generator=g, device="cuda")).to(torch.bfloat16)
               for _ in range(2)]
    return (parts if fused else tuple(p.contiguous() for p in parts)), weights


def compare(got, want, rounding, floor=0.0):
    got, want = np.float64(got), np.float64(want)
    slack = F32 * np.abs(want).max(-1, keepdims=True)
    assert (np.abs(got - want) <= np.maximum(rounding * (np.abs(want) + slack), floor) + slack).all()


def run(cache, q, k, v, position, slot, rotary, weights, eps, out=None, **kw):
    out = torch.full_like(q, -77.0) if out is None else out
    dsp.dspark_rope_append(cache, q, k, v, i32(position), torch.tensor(slot, device="cuda"), rotary,
                           out, *weights, eps, **kw)
    torch.cuda.synchronize()
    return out


CASES = {  # rows, heads_q, heads, dim, page, rot, pairs, norms, order, fused
    "one_row": (1, 1, 1, 64, 16, 64, False, "qk", "token", True),
    "one_row_many_heads": (1, 40, 8, 128, 16, 128, False, "qk", "token", True),
    "halves": (21, 8, 2, 128, 32, 128, False, "qk", "head", True),
    "pairs": (13, 5, 3, 128, 16, 128, True, "qk", "padded", False),
    "half_a_head_pairs": (19, 6, 2, 128, 64, 64, True, "q", "token", True),
    "half_a_head_halves": (17, 3, 1, 64, 256, 32, False, "k", "head", False),
    "sixteen_values": (9, 2, 2, 128, 16, 16, False, "qk", "token", True),
    "norm_alone": (11, 7, 5, 64, 16, 0, False, "qk", "token", True),
    "rotation_alone": (14, 4, 4, 64, 32, 64, True, "", "token", True),
    "append_alone": (5, 3, 1, 128, 16, 0, True, "", "token", True),
}


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("name", CASES)
def test_matches_oracle(name, fp8):
    rows, heads_q, heads, dim, ps, rot, pairs, norms, order, fused = CASES[name]
    rng = np.random.default_rng(rows)
    n_pages = -(-rows // ps) + 2
    cache = make_cache(n_pages, ps, heads, dim, fp8, order, seed=rows)
    (q, k, v), weights = rows_case(rows, heads_q, heads, dim, rows + 1, fused, std=3.0)
    weights = [w if s in norms else None for w, s in zip(weights, "qk")]
    position = rng.integers(0, 5000, rows)
    slot = rng.permutation(n_pages * ps)[:rows]
    if rows > 4:
        position[2], slot[3] = -1, -1     # padding; a row without a place
    f = inv_freq(rot)
    ws = [None if w is None else host(w).astype(np.float64) for w in weights]
    ks, vs = (None if s is None else host(s).astype(np.float64) for s in (cache.k_scale, cache.v_scale))
    want_q, want_k, want_v = op.rope_append(
        host(q), host(k), host(v), position, slot, f, pairs, *ws, 1e-5, np.full(q.shape, -77.0),
        host(cache.k), host(cache.v), ks, vs)
    out = run(cache, q, k, v, position, slot, dsp.Rotary(f, pairs), weights, 1e-5)
    compare(host(out), want_q, 2.0 ** -8)
    np.testing.assert_array_equal(host(cache.v), want_v)
    if fp8:
        compare(host(cache.k), np.clip(want_k, -448, 448), 2.0 ** -4, 2.0 ** -10)
    else:
        compare(host(cache.k), want_k, 2.0 ** -8)


@pytest.mark.parametrize("rows", [300, 5000])
def test_many_rows_equal_each_row_alone(rows):
    # warps take whole rows, or parts of one where there are few: the same arithmetic
    heads_q, heads, dim, ps = 9, 3, 128, 16
    n_pages = -(-rows // ps)
    (q, k, v), weights = rows_case(rows, heads_q, heads, dim, 5)
    position = np.random.default_rng(0).integers(0, 100000, rows)
    rotary = dsp.Rotary(inv_freq(dim))
    caches = [make_cache(n_pages, ps, heads, dim, False, fill=0.0) for _ in range(2)]
    slot = np.arange(rows)
    out = run(caches[0], q, k, v, position, slot, rotary, weights, 1e-6)
    one = torch.empty_like(out)
    for m in list(range(0, rows, 97)) + [rows - 1]:
        run(caches[1], q[m:m + 1], k[m:m + 1], v[m:m + 1], position[m:m + 1], slot[m:m + 1], rotary,
            weights, 1e-6, out=one[m:m + 1])
        assert torch.equal(one[m], out[m])
        for a, b in ((caches[0].k, caches[1].k), (caches[0].v, caches[1].v)):
            assert torch.equal(a[m // ps, m % ps], b[m // ps, m % ps])


@pytest.mark.parametrize("pairs", [False, True])
def test_far_positions(pairs):
    # the angle is exact to 2^31 positions: here 64-bit products of integers say what it is
    dim, heads = 128, 1
    f = inv_freq(dim, 5e5)
    rotary = dsp.Rotary(f, pairs)
    position = np.array([0, 1, 999983, 2 ** 24 + 1, 2 ** 31 - 1])
    rows = len(position)
    (q, k, v), _ = rows_case(rows, 1, heads, dim, 3)
    cache = make_cache(1, 16, heads, dim, False, fill=0.0)
    out = host(run(cache, q, k, v, position, np.arange(rows), rotary, (None, None), 0.0))
    x = np.float64(host(q))[:, 0]
    for m, p in enumerate(position):
        for i in range(dim // 2):
            turn = int(rotary.turns[i]) * int(p) % 2 ** 64
            t = 2 * math.pi * (turn / 2.0 ** 64)
            a, b = (2 * i, 2 * i + 1) if pairs else (i, i + dim // 2)
            size = abs(x[m, a]) + abs(x[m, b])
            for at, want in ((a, x[m, a] * math.cos(t) - x[m, b] * math.sin(t)),
                             (b, x[m, b] * math.cos(t) + x[m, a] * math.sin(t))):
                assert abs(out[m, 0, at] - want) <= 2.0 ** -8 * abs(want) + 2.0 ** -17 * size
            # and the units of a turn are the frequency's
            assert abs(int(rotary.turns[i]) / 2.0 ** 64 - f[i] / (2 * math.pi)) <= 2.0 ** -53
    assert int(rotary.turns[0]) > 0


def test_in_place_and_on_another_stream():
    rows, dim = 40, 64
    (q, k, v), weights = rows_case(rows, 6, 2, dim, 8)
    rotary = dsp.Rotary(inv_freq(dim))
    caches = [make_cache(3, 16, 2, dim, False, fill=0.0) for _ in range(2)]
    position, slot = np.arange(rows), np.arange(rows)
    want = run(caches[0], q, k, v, position, slot, rotary, weights, 1e-6)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    run(caches[1], q, k, v, position, slot, rotary, weights, 1e-6, out=q, stream=s)
    assert torch.equal(q, want) and torch.equal(caches[0].k, caches[1].k)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_values_that_are_no_numbers(fp8):
    # V goes as dspark_kv_append takes it; what is not turned keeps infinities to itself
    dim, rows = 128, 3
    (q, k, v), weights = rows_case(rows, 2, 2, dim, 9, fused=False)
    v[0, 0, :3] = torch.tensor([math.inf, -math.inf, math.nan])
    q[1, 1, 70] = math.inf       # not turned (rot 64), and no norm
    q[2, 0, 3] = math.nan
    caches = [make_cache(1, 16, 2, dim, fp8, fill=0.0, scales=False) for _ in range(2)]
    out = run(caches[0], q, k, v, [3, 4, 5], [0, 1, 2], dsp.Rotary(inv_freq(64)), (None, weights[1]),
              1e-6)
    dsp.dspark_kv_append(caches[1], k, v, torch.tensor([0, 1, 2], device="cuda"))
    raw = torch.uint8 if fp8 else torch.int16
    assert torch.equal(caches[0].v.view(raw), caches[1].v.view(raw))
    got = host(out)
    assert got[1, 1, 70] == math.inf and np.isfinite(np.delete(got[1, 1], 70)).all()
    assert np.isnan(got[2, 0, [3, 35]]).all() and np.isfinite(np.delete(got[2, 0], [3, 35])).all()
    assert np.isfinite(got[0]).all() and np.isfinite(got[1, 0]).all()


def test_slots_outside_the_cache():
    (q, k, v), weights = rows_case(3, 2, 2, 64, 4)
    cache = make_cache(2, 16, 2, 64, False, seed=3)
    before = host(cache.k), host(cache.v)
    out = run(cache, q, k, v, [1, 2, 3], [32, -5, 1 << 40], dsp.Rotary(inv_freq(64)), weights, 1e-6)
    assert dsp.dspark_device_status() == 9
    np.testing.assert_array_equal(host(cache.k), before[0])
    np.testing.assert_array_equal(host(cache.v), before[1])
    assert (out != -77).any(-1).all()      # the queries are turned all the same


@pytest.mark.parametrize("scale", [0.02, 0.25, 1.0, 3e-30, 1e30])
def test_e4m3_scales(scale):
    # without norm and rotation a key is stored as dspark_kv_append stores it, bit by bit
    rows, dim = 64, 128
    (q, k, v), _ = rows_case(rows, 1, 2, dim, 12, std=4.0 * min(scale, 1e3))
    raw = [torch.zeros((4, 16, 2, dim), device="cuda").to(torch.float8_e4m3fn) for _ in range(4)]
    scales = [torch.full((2,), scale, device="cuda") for _ in range(2)]
    a, b = dsp.KVCache(raw[0], raw[1], *scales), dsp.KVCache(raw[2], raw[3], *scales)
    slot = np.random.default_rng(1).permutation(rows)
    run(a, q, k, v, np.arange(rows), slot, dsp.Rotary([]), (None, None), 0.0)
    dsp.dspark_kv_append(b, k, v, torch.tensor(slot, device="cuda"))
    for x, y in ((a.k, b.k), (a.v, b.v)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
