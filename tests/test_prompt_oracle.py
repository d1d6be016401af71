"""The oracle of a prompt's way into the cache, pinned by closed forms and small cases."""
import math

import numpy as np

from oracle import cache as oc
from oracle import prompt as op


def test_rotation_keeps_lengths_and_depends_on_distance():
    rng = np.random.default_rng(0)
    f = 1e4 ** (-np.arange(8) / 8.0)
    for pairs in (False, True):
        q, k = rng.normal(size=(2, 24))
        dots = []
        for p in (0, 5, 1000):
            a = op.norm_rotate(q, None, 0.0, f, pairs, p + 7)
            b = op.norm_rotate(k, None, 0.0, f, pairs, p)
            assert np.allclose((a ** 2).sum(), (q ** 2).sum()) and (a[16:] == q[16:]).all()
            dots.append(a @ b)
        assert np.allclose(dots, dots[0], atol=1e-9)
    assert np.array_equal(op.norm_rotate(q, None, 0.0, f, True, 0), q)
    # a quarter turn
    got = op.norm_rotate([1.0, 2.0, 3.0, 4.0], None, 0.0, [math.pi / 2, 0.0], False, 1)
    assert np.allclose(got, [-3.0, 2.0, 1.0, 4.0])
    got = op.norm_rotate([1.0, 2.0, 3.0, 4.0], None, 0.0, [math.pi / 2, 0.0], True, 1)
    assert np.allclose(got, [-2.0, 1.0, 3.0, 4.0])


def test_norm():
    x = op.norm_rotate([3.0, 4.0], np.array([1.0, 2.0]), 0.0, [], False, 9)
    assert np.allclose(x, np.array([3.0, 8.0]) / math.sqrt(12.5))


def test_chunks_are_the_tree_oracles_chains():
    rng = np.random.default_rng(1)
    k, v = rng.normal(size=(2, 6, 16, 2, 8))
    q = rng.normal(size=(9, 4, 8))
    args = (np.array([20, 3]), np.array([0, 5, 9]), np.array([[4, 1], [0, 5]]), 0.3)
    out, lse, size = op.chunk_attention(q, k, v, *args, np.array([0.5, 2.0]), np.array([3.0, 0.1]))
    want, want_lse = oc.tree_attention(q, k, v, *args[:2], None, *args[2:], np.array([0.5, 2.0]),
                                       np.array([3.0, 0.1]))
    assert np.allclose(out, want) and np.allclose(lse, want_lse) and (size >= np.abs(out) - 1e-12).all()


def test_a_forks_life():
    p = dict(ctx=np.array([33, -1, -1]), held=np.array([3, 0, 0]), n_free=2,
             free_pages=np.array([1, 2, 0, 0, 0]), block_table=np.array([[4, 3, 0], [-1] * 3, [-1] * 3]),
             refs=np.zeros(5, dtype=int))
    a = op.kv_fork([0, 0], [1, 2], 16, **p)
    assert a["copies"].tolist() == [[0, 2, 1], [0, 1, 1]] and a["n_free"] == 0
    assert a["block_table"].tolist() == [[4, 3, 0], [4, 3, 2], [4, 3, 1]]
    assert a["refs"].tolist() == [0, 0, 0, 2, 2]
    p.update({k: a[k] for k in ("ctx", "held", "n_free", "block_table", "refs")})
    p["ctx"] = np.array([-1, 33, -1])
    p.update(op.kv_release(**p))
    assert p["free_pages"][:2].tolist() == [0, 1] and p["refs"].tolist() == [0] * 5 and p["n_free"] == 2
    p["ctx"][1] = -1
    p.update(op.kv_release(**p))
    assert p["free_pages"].tolist() == [0, 1, 4, 3, 2] and p["n_free"] == 5


def test_squeezing():
    got = op.kv_squeeze(held=np.array([2, 1]), n_free=3, free_pages=np.array([2, 5, 0, 9, 9, 9]),
                        block_table=np.array([[3, 1], [4, 7]]), refs=np.array([0, 1, 0, 0, 2, 0]))
    assert got["move_from"].tolist() == [3, 4, -1] and got["move_to"].tolist() == [0, 2, -1]
    assert got["block_table"].tolist() == [[0, 1], [2, 7]] and got["refs"].tolist() == [0, 1, 2, 0, 0, 0]
    assert got["free_pages"].tolist() == [5, 4, 3, 9, 9, 9]
    assert got["new_page"].tolist() == [-1, 1, -1, 0, 2, -1] and got["n_moves"] == 2
    cache = np.arange(6.0).reshape(6, 1, 1, 1)
    moved = op.kv_copy(cache, got["move_from"], got["move_to"]).ravel()
    assert moved[:3].tolist() == [3, 1, 4]
