"""Places of a shared pool that are forked into as soon as they are left, with no plan and no
release between: their pages go back, and are there for the forks."""
import numpy as np
import pytest
import torch

from test_gpu_cache import dsp, host, i32, _lib  # noqa: F401
from test_gpu_prompt_pool import PAGE, TYPES, caches_of, make_pool, rotary, step, tokens_of

pytestmark = pytest.mark.gpu


@TYPES
def test_a_place_that_was_just_left_is_forked_into(fp8):
    lengths = [70, 150, 33, 90]
    # as many pages as the requests hold: a fork's own page is one of those that come back
    pool = make_pool(R=4, pages=sum(-(-n // PAGE) for n in lengths), shared=True)
    caches, rot = caches_of(pool, fp8), rotary()
    pool.ctx.zero_()
    step(pool, caches, lengths, rot, 1)
    pool.commit(i32(lengths))
    assert int(pool.n_free) == 0
    before = [tokens_of(pool, c) for c in caches]
    pool.ctx[2:] = -1
    pool.fork(i32([0, 1]), i32([3, 2]))
    for c in caches:
        pool.copy(c)
    assert dsp.dspark_device_status() == 0
    assert host(pool.ctx).tolist() == [70, 150, 150, 70]
    for c, b in zip(caches, before):
        after = tokens_of(pool, c)
        for child, of in ((0, 0), (1, 1), (2, 1), (3, 0)):
            np.testing.assert_array_equal(after[child], b[of])
    step(pool, caches, [5, 1, 20, 70], rot, 2)      # they go on, each with pages of its own
    pool.commit(i32([5, 1, 20, 70]))
    for c, b in zip(caches, before):
        after = tokens_of(pool, c)
        for child, of in ((0, 0), (1, 1), (2, 1), (3, 0)):
            np.testing.assert_array_equal(after[child][:len(b[of])], b[of])
    pool.ctx.fill_(-1)
    pool.release()
    assert sorted(host(pool.free_pages)) == list(range(len(pool.free_pages)))
    assert int(pool.n_free) == len(pool.free_pages) and not pool.refs.any()
    assert dsp.dspark_device_status() == 0


@TYPES
def test_places_left_and_forked_into_in_a_graph(fp8):
    # captured once; between replays the samples end by their ctx alone
    pool = make_pool(R=3, pages=40, shared=True)
    caches, rot = caches_of(pool, fp8, 1), rotary()
    pool.ctx[0] = 0
    step(pool, caches, [77, 0, 0], rot, 1)
    pool.commit(i32([77, 0, 0]))
    before = tokens_of(pool, caches[0])[0]
    source, target = i32([0, 0]), i32([1, 2])

    def body():
        pool.fork(source, target)
        pool.copy(caches[0])

    body()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        body()
    free = None
    for _ in range(4):
        pool.ctx[1:] = -1
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert host(pool.ctx).tolist() == [77] * 3
        for tokens in tokens_of(pool, caches[0]):
            np.testing.assert_array_equal(tokens, before)
        assert free in (None, int(pool.n_free))
        free = int(pool.n_free)
    assert dsp.dspark_device_status() == 0
