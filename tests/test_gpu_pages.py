"""Pages with several holders against the plain oracle: whole numbers and copies, all equal."""
import numpy as np
import pytest
import torch

from oracle import prompt as op
from test_gpu_cache import dsp, host, i32, make_cache, _lib  # noqa: F401

pytestmark = pytest.mark.gpu


def pool(rng, R, ps, max_pages, n_pages, live, longest):
    """Tables of R places of which `live` hold pages of their own."""
    ctx = np.full(R, -1)
    ctx[rng.permutation(R)[:live]] = rng.integers(0, longest + 1, live)
    held = np.where(ctx >= 0, np.minimum(-(-ctx // ps) + rng.integers(0, 2, R), max_pages), 0)
    order = rng.permutation(n_pages)
    table = np.full((R, max_pages), -1)
    at = 0
    for r in range(R):
        table[r, :held[r]] = order[at:at + held[r]]
        at += held[r]
    free = np.concatenate([order[at:], order[:at]])
    return dict(ctx=ctx, held=held, n_free=n_pages - at, free_pages=free, block_table=table,
                refs=np.zeros(n_pages, dtype=np.int64))


def on_gpu(p):
    return {k: i32([v] if k == "n_free" else v) for k, v in p.items()}


def check(t, p, names):
    for k in names:
        np.testing.assert_array_equal(host(t[k]), np.asarray([p[k]] if k == "n_free" else p[k]), k)


def fork(t, source, target, ps):
    n = len(source)
    copies = [torch.full((n,), -9, dtype=torch.int32, device="cuda") for _ in range(3)]
    dsp.dspark_kv_fork(i32(source), i32(target), ps, t["ctx"], t["held"], t["n_free"],
                       t["free_pages"], t["block_table"], t["refs"], *copies)
    return np.stack([host(c) for c in copies], 1)


def release(t):
    dsp.dspark_kv_release(t["ctx"], t["held"], t["n_free"], t["free_pages"], t["block_table"],
                          t["refs"])


TABLES = ["ctx", "held", "n_free", "block_table", "refs"]
SIZES = [  # R, page, live, longest context
    (2, 16, 1, 40), (9, 16, 3, 100), (33, 32, 20, 200), (200, 16, 40, 700), (1500, 64, 100, 1000),
    (16384, 16, 300, 60)]


@pytest.mark.parametrize("R,ps,live,longest", SIZES)
def test_forks_then_releases(R, ps, live, longest):
    rng = np.random.default_rng(R + ps)
    most = -(-longest // ps) + 2
    p = pool(rng, R, ps, most, live * most + 3 * R, live, longest)
    t = on_gpu(p)
    for step in range(3):
        there, away = np.flatnonzero(p["ctx"] >= 0), np.flatnonzero(p["ctx"] < 0)
        n = max(1, min(len(away) * 2 // 3, R))
        if len(there) and len(away):
            source = rng.choice(there, n)
            source[rng.random(n) < 0.1] = -1    # no fork
            target = rng.permutation(away)[:n]
            want = op.kv_fork(source, target, ps, **p)
            got = fork(t, source, target, ps)
            np.testing.assert_array_equal(got, want["copies"])
            p.update({k: want[k] for k in TABLES})
            check(t, p, TABLES)
            assert not want["bad"] and not want["starved"]
        left = rng.random(R) < 0.5              # sources among them
        p["ctx"] = np.where(left, -1, p["ctx"])
        t["ctx"] = i32(p["ctx"])
        p.update(op.kv_release(**p))
        release(t)
        check(t, p, TABLES + ["free_pages"])
        assert len(set(p["free_pages"][:p["n_free"]])) == p["n_free"]
    p["ctx"][:] = -1
    t["ctx"].fill_(-1)
    release(t)
    assert int(t["n_free"]) == len(p["free_pages"]) and not t["refs"].any()
    release(t)                                  # nobody is left
    assert int(t["n_free"]) == len(p["free_pages"])
    assert dsp.dspark_device_status() == 0


def test_a_page_whose_holders_leave_one_after_the_other():
    p = dict(ctx=np.array([40, -1, -1, -1]), held=np.array([3, 0, 0, 0]), n_free=5,
             free_pages=np.array([0, 1, 2, 3, 4, 9, 9, 9]),
             block_table=np.array([[7, 5, 6], [-1] * 3, [-1] * 3, [-1] * 3]),
             refs=np.zeros(8, dtype=np.int64))
    t = on_gpu(p)
    copies = fork(t, [0, 0, 0], [2, 1, 3], 16)
    assert copies.tolist() == [[6, 4, 8], [6, 3, 8], [6, 2, 8]]
    assert host(t["refs"]).tolist() == [0, 0, 0, 0, 0, 3, 0, 3]
    for left, free in ((0, [0, 1, 6]), (3, [0, 1, 6, 2]), (1, [0, 1, 6, 2, 3])):
        t["ctx"][left] = -1
        release(t)
        assert host(t["free_pages"])[:int(t["n_free"])].tolist() == free
    t["ctx"][2] = -1
    release(t)
    assert host(t["free_pages"]).tolist() == [0, 1, 6, 2, 3, 7, 5, 4] and not t["refs"].any()


@pytest.mark.parametrize("R", [8, 100])
def test_forks_that_are_refused(R):
    ps, n_pages = 16, 64
    ctx, held = np.full(R, -1), np.zeros(R, dtype=np.int64)
    table = np.full((R, 4), -1)
    ctx[0], held[0], table[0, :2] = 20, 2, [3, 4]
    ctx[1], held[1], table[1, :1] = 20, 1, [5]      # holds fewer pages than it has tokens for
    held[2], table[2, 0] = 1, 6                     # left, but not released
    p = dict(ctx=ctx, held=held, n_free=40, free_pages=np.arange(n_pages), block_table=table,
             refs=np.zeros(n_pages, dtype=np.int64))
    extra = [-1] * (40 if R == 100 else 0)
    source = [0, 1, 0, 3, 0, 0, 0, 0] + extra
    target = [4, 5, 2, 5, 4, R, 6, 1] + [7] * len(extra)
    want = op.kv_fork(source, target, ps, **p)
    t = on_gpu(p)
    np.testing.assert_array_equal(fork(t, source, target, ps), want["copies"])
    assert dsp.dspark_device_status() == 1 and want["bad"] == 6
    check(t, dict(p, **{k: want[k] for k in TABLES}), TABLES)


@pytest.mark.parametrize("n_free", [0, 1, 3])
def test_forks_without_pages(n_free):
    # the first one in need without a page ends the giving; whole pages need none
    p = dict(ctx=np.array([20, 32, -1, -1, -1, -1, -1, -1]), held=np.array([2, 2] + [0] * 6),
             n_free=n_free, free_pages=np.arange(32),
             block_table=np.concatenate([[[30, 31], [28, 29]], np.full((6, 2), -1)]),
             refs=np.zeros(32, dtype=np.int64))
    source, target = [0, 1, 0, 0, 1], [2, 3, 4, 5, 6]
    want = op.kv_fork(source, target, 16, **p)
    t = on_gpu(p)
    np.testing.assert_array_equal(fork(t, source, target, 16), want["copies"])
    assert dsp.dspark_device_status() == (9 if want["starved"] else 0)
    check(t, dict(p, **{k: want[k] for k in TABLES}), TABLES)


def test_tables_that_are_not_sound_are_reported():
    t = on_gpu(dict(ctx=[-1, -1], held=[2, 1], n_free=1, free_pages=[0, 1, 2, 3],
                    block_table=[[9, 1], [1, -1]], refs=[0, 0, 0, 0]))
    release(t)                                   # a page outside the cache, one held once too often
    assert dsp.dspark_device_status() == 9
    assert host(t["n_free"]).tolist() == [2] and host(t["free_pages"]).tolist()[:2] == [0, 1]
    t = on_gpu(dict(ctx=[-1], held=[-3], n_free=9, free_pages=[0, 1], block_table=[[0]], refs=[0, 0]))
    release(t)
    assert dsp.dspark_device_status() == 9


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("R,n_pages,part", [(1, 2, 0.5), (3, 16, 0.4), (8, 97, 0.9), (40, 1000, 0.1),
                                            (40, 1025, 0.5), (700, 9001, 0.6), (5, 64, 0.0),
                                            (5, 64, 1.0)])
def test_squeeze(R, n_pages, part, in_place):
    rng = np.random.default_rng(n_pages)
    used = int(n_pages * part)
    order = rng.permutation(n_pages)
    cut = np.sort(rng.integers(0, used + 1, R - 1))
    held = np.diff(np.concatenate([[0], cut, [used]]))
    table = np.full((R, held.max() + 2), -1)
    at = 0
    for r in range(R):
        table[r, :held[r]] = order[at:at + held[r]]
        at += held[r]
    refs = np.zeros(n_pages, dtype=np.int64)
    for r in range(1, R):                        # a page of the request before, too
        if held[r - 1] and r % 2:
            table[r, held[r]] = table[r - 1, 0]
            held[r] += 1
            refs[table[r - 1, 0]] += 1
    p = dict(held=held, n_free=n_pages - used, free_pages=np.concatenate([order[used:], order[:used]]),
             block_table=table, refs=refs)
    want = op.kv_squeeze(**p)
    t = on_gpu(p)
    new = lambda *n: torch.full(n, -9, dtype=torch.int32, device="cuda")  # noqa: E731
    outs = ([t["free_pages"], t["block_table"], t["refs"]] if in_place else
            [new(n_pages), new(*table.shape), new(n_pages)])
    rest = [new(n_pages), new(n_pages // 2), new(n_pages // 2), new(1)]
    dsp.dspark_kv_squeeze(t["held"], t["n_free"], t["free_pages"], t["block_table"], t["refs"], *outs,
                          *rest)
    for got, name in zip(outs + rest, ["free_pages", "block_table", "refs", "new_page", "move_from",
                                       "move_to", "n_moves"]):
        np.testing.assert_array_equal(host(got), np.atleast_1d(want[name]), name)
    assert dsp.dspark_device_status() == 0


def test_squeeze_of_a_stack_that_is_not_sound():
    held, table = i32([1]), i32([[5]])
    new = lambda *n: torch.full(n, -9, dtype=torch.int32, device="cuda")  # noqa: E731
    for free in ([0, 0, 1, 2, 3, 4], [0, 9, 1, 2, 3, 4], [-1, 2, 1, 0, 3, 4]):
        dsp.dspark_kv_squeeze(held, i32([2]), i32(free), table, i32([0] * 6), new(6), new(1, 1), new(6),
                              new(6), new(3), new(3), new(1))
        assert dsp.dspark_device_status() == 9


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("heads,dim,ps,order,n", [
    (1, 64, 16, "token", 1), (2, 64, 16, "head", 7), (5, 128, 32, "padded", 40),
    (8, 128, 64, "token", 300), (40, 128, 16, "token", 5), (8, 64, 256, "head", 9)])
def test_copies(heads, dim, ps, order, n, fp8):
    rng = np.random.default_rng(heads + ps)
    n_pages = 2 * n + 3
    cache = make_cache(n_pages, ps, heads, dim, fp8, order, seed=n)
    order_ = rng.permutation(n_pages)
    a, b = order_[:n], order_[n:2 * n]
    a = np.where(rng.random(n) < 0.2, -1, a)
    for tokens in (None, rng.integers(0, ps + 1, n)):
        want = [op.kv_copy(host(x), a, b, tokens) for x in (cache.k, cache.v)]
        dsp.dspark_kv_copy(cache, i32(a), i32(b), None if tokens is None else i32(tokens))
        for x, w in zip((cache.k, cache.v), want):
            np.testing.assert_array_equal(host(x), w)
        a, b = np.where(a < 0, -1, b), np.where(a < 0, b, a)  # and back, into the other ones
    assert dsp.dspark_device_status() == 0


def test_copies_outside_the_cache():
    cache = make_cache(4, 16, 2, 64, False, seed=1)
    before = host(cache.k), host(cache.v)
    for a, b, n, rc in (([4], [0], [1], 9), ([0], [4], [1], 9), ([0], [-1], [1], 9), ([0], [1], [17], 6),
                        ([0], [1], [-1], 6), ([-7], [99], [99], 0)):
        dsp.dspark_kv_copy(cache, i32(a), i32(b), i32(n))
        assert dsp.dspark_device_status() == rc, (a, b, n)
    np.testing.assert_array_equal(host(cache.k), before[0])
    np.testing.assert_array_equal(host(cache.v), before[1])
    dsp.dspark_kv_copy(cache, i32([]), i32([]))
