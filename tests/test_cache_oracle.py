"""Pins of the paged-cache oracle: hand-worked cases and closed forms (CPU)."""
import math

import numpy as np

from oracle import cache as oc


def test_e4m3_values_and_rounding():
    v = oc.e4m3_values()
    assert v[0x7e] == 448.0 and v[0x08] == 2.0 ** -6 and v[0x01] == 2.0 ** -9 and np.isnan(v[0x7f])
    # 17 lies halfway between 16 and 18: to the even code; 1000 saturates
    x = oc.e4m3_round(np.array([17.0, 19.0, 1000.0, -0.3, 2.0 ** -10, np.nan, 1.5 * 2.0 ** -9]))
    np.testing.assert_array_equal(x[:5], [16.0, 20.0, 448.0, -0.3125, 0.0])
    assert np.isnan(x[5]) and x[6] == 2.0 ** -8


def test_plan_by_hand():
    # request 0 grows into a new page, 1 has left with two pages, 2 has room
    out = oc.kv_plan(ctx=[15, -1, 3], length=[2, 9, 1], extra=1, parent=[[0, 0], [0, 0], [0, 0]],
                     page_size=16, held=[1, 2, 1], n_free=1, free_pages=[5, 0, 0, 0],
                     block_table=[[7, 0], [2, 3], [4, 0]], n_rows=8)
    assert out["row_start"].tolist() == [0, 3, 3, 5]
    assert out["free_pages"].tolist() == [5, 2, 3, 0] and out["n_free"] == 2
    assert out["block_table"].tolist() == [[7, 3], [2, 3], [4, 0]]
    assert out["held"].tolist() == [2, 0, 1]
    assert out["slot"].tolist() == [7 * 16 + 15, 48, 49, 67, 68, -1, -1, -1]
    assert out["position"].tolist() == [15, 16, 16, 3, 4, -1, -1, -1]
    assert out["anc"].tolist() == [1, 3, 5, 1, 3, 0, 0, 0]


def test_plan_without_pages_starves_later_needs_only():
    out = oc.kv_plan(ctx=[0, 16, 0], length=[16, 15, 1], extra=0, parent=None, page_size=16,
                     held=[0, 1, 1], n_free=0, free_pages=[9], block_table=[[8, 8], [1, 8], [2, 8]], n_rows=32)
    assert out["block_table"].tolist() == [[-1, 8], [1, -1], [2, 8]]
    assert out["held"].tolist() == [0, 1, 1] and out["n_free"] == 0
    assert (out["slot"][:31] == -1).all() and out["slot"][31] == 32


def test_attention_closed_forms():
    # equal keys: the mean of the visible values, lse = s + log(count)
    k = np.zeros((3, 16, 1, 4))
    v = np.arange(3 * 16 * 4, dtype=float).reshape(3, 16, 1, 4)
    k[..., 0] = 2.0
    q = np.zeros((2, 2, 4))
    q[..., 0] = 3.0
    out, lse = oc.tree_attention(q, k, v, [17], [0, 2], np.array([1, 2], np.uint64),
                                 np.array([[2, 0]]), 0.5)
    ctx = [(2, t) for t in range(16)] + [(0, 0)]
    for i, node in enumerate([(0, 1), (0, 2)]):
        want = np.mean([v[p, t, 0] for p, t in ctx + [node]], 0)
        np.testing.assert_allclose(out[i], np.stack([want, want]))
        np.testing.assert_allclose(lse[i], 3.0 + math.log(18))
    # nothing visible
    out, lse = oc.tree_attention(q[:1], k, v, [0], [0, 1], np.array([0], np.uint64),
                                 np.array([[1]]), 0.5)
    assert (out == 0).all() and (lse == -math.inf).all()


def test_accept_and_compact_by_hand():
    # node 0 -> 1, 2; 2 -> 3, 4: the target wants 20 after the anchor, 40 after node 2
    acc, bonus, paths, ctx = oc.tree_accept([0, 5], [[0, 0, 2, 2]], [[10, 20, 30, 40]],
                                            [20, 0, 40, 0, 99], [6])
    assert (acc, bonus, paths, ctx) == ([2], [99], [[2, 4]], [9])
    cache = np.arange(32.0).reshape(2, 16, 1, 1)
    out = oc.kv_compact(cache, [14], paths, np.array([[1, 0]]))
    # position 15 (page 1) takes 16 (page 0), position 16 takes 18
    assert out[1, 15, 0, 0] == 0 and out[0, 0, 0, 0] == 2
    # two matching children: the lower; a chain stops at the first miss
    assert oc.tree_accept([0, 3], [[0, 0]], [[5, 5]], [5, 1, 2], [0])[2] == [[1]]
    assert oc.tree_accept([0, 4], None, [[1, 2, 3]], [1, 2, 9, 4], [0])[:3] == ([2], [9], [[1, 2]])


def test_append_rounds_the_quotient():
    cache = np.zeros((1, 16, 2, 1))
    out = oc.kv_append(cache, np.array([[[1.0], [1.0]], [[5.0], [5.0]]]), [3, -1], [0.5, 0.1])
    assert out[0, 3, 0, 0] == 2.0 and out[0, 3, 1, 0] == 10.0 and np.count_nonzero(out) == 2
