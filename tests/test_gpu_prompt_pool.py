"""A prompt's way into the cache as it is used: PagePool with rotation, chunks, forks, rounds
over forked requests, releases and squeezing, in order and in captured graphs.  The
attention is held to the float64 oracle with the tolerances of test_gpu_chunk, over what
the caches hold; pages are compared token by token with what they were."""
import numpy as np
import pytest
import torch

from oracle import prompt as op
from test_gpu_cache import dsp, host, i32, make_cache, _lib  # noqa: F401
from test_gpu_chunk import check

pytestmark = pytest.mark.gpu

TYPES = pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
HEADS, GROUP, DIM, PAGE = 2, 4, 64, 16
HEADS_Q = HEADS * GROUP


def normal(shape, seed, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (std * torch.randn(shape, generator=g, device="cuda")).to(torch.bfloat16)


def make_pool(R=8, rows=600, pages=200, tokens=1000, **kw):
    return dsp.PagePool(R, pages, PAGE, tokens, rows, **kw)


def rotary():
    return dsp.Rotary(1e4 ** (-np.arange(DIM // 2) * 2.0 / DIM))


def step(pool, caches, ns, rot, seed, extra=0, fp8=False):
    """Plans ns new rows a request, rotates, appends and attends in every layer, and compares
    each layer's attention with the oracle over the layer's cache."""
    ctx = host(pool.ctx).copy()
    pool.plan(i32(np.array(ns) - extra), extra=extra)
    rows, outs = pool.n_rows, []
    total = int(sum(n for n, c in zip(ns, ctx) if c >= 0))
    for layer, cache in enumerate(caches):
        qkv = normal((rows, HEADS_Q + 2 * HEADS, DIM), 100 * seed + layer, 1.5)
        weights = [normal((DIM,), 7 + i) for i in range(2)]
        q, k, v = qkv[:, :HEADS_Q], qkv[:, HEADS_Q:HEADS_Q + HEADS], qkv[:, HEADS_Q + HEADS:]
        pool.rope_append(cache, q, k, v, rot, q, *weights)
        out = torch.full((rows, HEADS_Q, DIM), -77.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((rows, HEADS_Q), -77.0, device="cuda")
        pool.attend(cache, q, max(max(ns), 1), out, lse)
        case = dict(cache=cache, q=q, ctx=np.maximum(ctx, 0), row_start=host(pool.row_start),
                    table=host(pool.block_table), scale=DIM ** -0.5)
        check(case, out, lse)
        outs.append(out[:total].clone())
    return outs


def tokens_of(pool, cache):
    """Every request's committed K, in order."""
    table, ctx = host(pool.block_table), host(pool.ctx)
    k = host(cache.k)
    return [np.stack([k[table[r, p // PAGE], p % PAGE] for p in range(c)]) if c > 0 else None
            for r, c in enumerate(ctx)]


def caches_of(pool, fp8, layers=2):
    return [make_cache(len(pool.free_pages), PAGE, HEADS, DIM, fp8, fill=0.0, seed=50 + i)
            for i in range(layers)]


@TYPES
def test_prompts_chunks_forks_rounds_and_squeezing(fp8):
    pool = make_pool(shared=True)
    caches, rot = caches_of(pool, fp8), rotary()
    pool.ctx[:3] = 0
    none = [0] * 5
    step(pool, caches, [200, 37, 300] + none, rot, 1)       # prompts, one of few rows
    pool.commit(i32([200, 37, 300] + none))
    step(pool, caches, [133, 1, 90] + none, rot, 2)         # their next chunks
    pool.commit(i32([133, 1, 90] + none))
    before = [tokens_of(pool, c) for c in caches]
    pool.fork(i32([0, 0, 2, -1, 1]), i32([5, 3, 7, 4, 6]))
    for c in caches:
        pool.copy(c)
    assert host(pool.ctx).tolist() == [333, 38, 390, 333, -1, 333, 38, 390]
    for c, b in zip(caches, before):
        after = tokens_of(pool, c)
        for child, of in ((3, 0), (5, 0), (6, 1), (7, 2)):
            np.testing.assert_array_equal(after[child], b[of])
    # a round each, all of them over shared pages: drafts differ, the past does not
    step(pool, caches, [3, 2, 6, 1, 0, 4, 5, 6], rot, 3, extra=1)
    pool.commit(i32([2, 1, 6, 1, 0, 3, 1, 4]))
    for c, b in zip(caches, before):
        after = tokens_of(pool, c)
        for child, of in ((0, 0), (3, 0), (5, 0), (1, 1), (6, 1), (2, 2), (7, 2)):
            np.testing.assert_array_equal(after[child][:len(b[of])], b[of])
    # the prompts themselves leave; their continuations go on
    free = int(pool.n_free)
    pool.ctx[:3] = -1
    step(pool, caches, [0, 0, 0, 70, 0, 65, 1, 90], rot, 4)
    pool.commit(i32([0, 0, 0, 70, 0, 65, 1, 90]))
    assert int(pool.refs.sum()) == 333 // PAGE              # requests 3 and 5 share the rest
    before = [tokens_of(pool, c) for c in caches]
    held = int(pool.held.sum()) - int(pool.refs.sum())
    pool.squeeze()
    for c in caches:
        pool.move(c)
    used = len(pool.free_pages) - int(pool.n_free)
    assert used == held and int(pool.block_table[pool.ctx >= 0].max()) < used <= len(pool.free_pages)
    for c, b in zip(caches, before):
        for x, y in zip(tokens_of(pool, c), b):
            assert (x is None) == (y is None)
            if x is not None:
                np.testing.assert_array_equal(x, y)
    step(pool, caches, [0, 0, 0, 5, 0, 80, 2, 1], rot, 5)
    pool.ctx.fill_(-1)
    pool.release()
    assert int(pool.n_free) == len(pool.free_pages) and not pool.refs.any()
    assert sorted(host(pool.free_pages)) == list(range(len(pool.free_pages))) and free >= 0
    assert dsp.dspark_device_status() == 0


@TYPES
def test_forks_and_their_chunks_in_a_graph(fp8):
    # captured once, replayed with other places and lengths: fork, copy, plan, rotate, attend
    pool = make_pool(R=4, shared=True)
    caches, rot = caches_of(pool, fp8, 1), rotary()
    cache = caches[0]
    pool.ctx[:2] = 0
    step(pool, caches, [70, 150, 0, 0], rot, 1)
    pool.commit(i32([70, 150, 0, 0]))
    source, target, new = i32([-1, -1]), i32([2, 3]), i32([0, 0, 0, 0])
    qkv = normal((pool.n_rows, HEADS_Q + 2 * HEADS, DIM), 9)
    q = torch.empty((pool.n_rows, HEADS_Q, DIM), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.zeros_like(q), torch.zeros((pool.n_rows, HEADS_Q), device="cuda")

    def body():
        pool.fork(source, target)
        pool.copy(cache)
        pool.plan(new, extra=0)
        pool.rope_append(cache, qkv[:, :HEADS_Q], qkv[:, HEADS_Q:HEADS_Q + HEADS],
                         qkv[:, HEADS_Q + HEADS:], rot, q)
        pool.attend(cache, q, 200, out, lse)

    body()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        body()
    for forks, ns in (([0, 1], [1, 90, 66, 5]), ([1, 0], [3, 0, 120, 101]), ([-1, 1], [100, 1, 0, 65])):
        pool.ctx[2:] = -1
        pool.release()
        source.copy_(i32(forks))
        new.copy_(i32(ns))
        out.fill_(-77.0)
        lse.fill_(-77.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want = [70, 150] + [(70, 150)[f] if f >= 0 else -1 for f in forks]
        assert host(pool.ctx).tolist() == want
        case = dict(cache=cache, q=q, ctx=np.maximum(want, 0), row_start=host(pool.row_start),
                    table=host(pool.block_table), scale=DIM ** -0.5)
        check(case, out, lse)
    assert dsp.dspark_device_status() == 0


def test_a_pool_without_sharing_takes_long_prompts():
    pool = make_pool(R=3)
    caches, rot = caches_of(pool, False), rotary()
    pool.ctx.zero_()
    step(pool, caches, [400, 10, 150], rot, 1)
    pool.commit(i32([400, 10, 150]))
    step(pool, caches, [64, 1, 3], rot, 2)      # few rows: the tree attention's chains
    assert dsp.dspark_device_status() == 0


def test_two_streams_attend_chunks_at_once():
    pool = make_pool(R=3, pages=400, tokens=3000, rows=2500)
    caches, rot = caches_of(pool, False), rotary()
    pool.ctx.zero_()
    ns = [900, 700, 800]
    pool.plan(i32(ns), extra=0)
    qs = [normal((pool.n_rows, HEADS_Q, DIM), 40 + i) for i in range(2)]
    for i, c in enumerate(caches):
        kv = normal((pool.n_rows, 2 * HEADS, DIM), 60 + i)
        pool.append(c, kv[:, :HEADS], kv[:, HEADS:])
    want = [torch.zeros_like(q) for q in qs]
    for c, q, o in zip(caches, qs, want):
        pool.attend(c, q, 900, o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[torch.zeros_like(q) for _ in range(10)] for q in qs]
    torch.cuda.synchronize()
    for k in range(10):
        for i, s in enumerate(streams):
            pool.attend(caches[i], qs[i], 900, got[i][k], stream=s)
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])
