"""PagePool on the GPU: a prompt's rows after a tree's, calls on several streams, and
whole rounds in a captured graph.  The attention is held to the
float64 oracle with the tolerances of test_gpu_cache."""
import numpy as np
import pytest
import torch

from oracle import cache as oc
from test_gpu_cache import check_attention, dsp, host, i32, make_cache, _lib  # noqa: F401

pytestmark = pytest.mark.gpu

TYPES = pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
HEADS, GROUP, DIM, PAGE = 2, 4, 64, 16


def normal(shape, seed, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (std * torch.randn(shape, generator=g, device="cuda")).to(torch.bfloat16)


def make_pool(R=3, rows=96):
    pool = dsp.PagePool(R, 64, PAGE, 256, rows)
    pool.ctx.zero_()
    return pool


def as_case(pool, cache, q, ns, ctx, anc):
    """What check_attention takes, from a pool after its plan."""
    return dict(cache=cache, q=q, ctx=np.array(ctx), ns=ns, anc=anc, scale=DIM ** -0.5,
                row_start=host(pool.row_start), table=host(pool.block_table))


@TYPES
def test_a_prompt_after_a_tree_round(fp8):
    # star-shaped trees leave masks that hide a row from the next; then a prompt of up to
    # 64 rows in the same pool, whose rows see all before them
    pool = make_pool()
    cache = make_cache(64, PAGE, HEADS, DIM, fp8, seed=1)
    rows = pool.n_rows
    pool.plan(i32([7, 7, 7]), parent=i32(np.zeros((3, 7))))
    pool.commit(i32([5, 0, 1]))
    ns, ctx = [20, 64, 9], [5, 0, 1]
    pool.plan(i32(ns), extra=0)
    pool.append(cache, normal((rows, HEADS, DIM), 2), normal((rows, HEADS, DIM), 3))
    q = normal((rows, HEADS * GROUP, DIM), 4)
    out = torch.full_like(q, -77.0)
    lse = torch.full((rows, HEADS * GROUP), -77.0, device="cuda")
    pool.attend(cache, q, 64, out, lse)
    check_attention(as_case(pool, cache, q, ns, ctx, None), out, lse)
    assert dsp.dspark_device_status() == 0


def long_contexts(layers, fp8, R=3, tokens=2500):
    """A pool whose requests hold contexts that are cut over many CTAs, and its layers."""
    n_pages = R * (tokens // PAGE + 2)
    pool = dsp.PagePool(R, n_pages, PAGE, tokens + 100, R * tokens)
    pool.ctx.zero_()
    pool.plan(i32([tokens] * R), extra=0)
    pool.commit(i32([tokens] * R))
    return pool, [make_cache(n_pages, PAGE, HEADS, DIM, fp8, seed=30 + i) for i in range(layers)]


@TYPES
def test_attends_on_two_streams_at_once(fp8):
    pool, caches = long_contexts(2, fp8)
    pool.plan(i32([7, 7, 7]))
    rows = pool.n_rows
    qs = [normal((rows, HEADS * GROUP, DIM), 40 + i) for i in range(2)]
    want = [torch.zeros_like(q) for q in qs]
    for cache, q, out in zip(caches, qs, want):
        pool.attend(cache, q, 8, out)
    torch.cuda.synchronize()
    assert not torch.equal(*want)
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[torch.zeros_like(q) for _ in range(20)] for q in qs]
    torch.cuda.synchronize()
    for k in range(20):
        for i, s in enumerate(streams):
            pool.attend(caches[i], qs[i], 8, got[i][k], stream=s)
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(out, want[i]) for out in got[i])


@TYPES
@pytest.mark.parametrize("tree", [False, True], ids=["chain", "tree"])
def test_a_whole_round_in_a_graph(tree, fp8):
    # plan, append, attend (two layers), accept and compact captured once and replayed from
    # several states, against direct calls
    gamma = 7
    pool, caches = long_contexts(2, fp8)
    rows, R = pool.n_rows, 3
    length = i32([7, 3, 5])
    parent = i32([[0, 0, 1, 2, 2, 4, 6], [0, 1, 0, 0, 0, 0, 0], [0, 1, 1, 3, 3, 0, 0]]) if tree \
        else None
    kv = normal((2, rows, 2 * HEADS, DIM), 50)
    q = normal((2, rows, HEADS * GROUP, DIM), 51)
    out, lse = torch.zeros_like(q), torch.zeros((2, rows, HEADS * GROUP), device="cuda")
    tokens = torch.zeros((R, gamma), dtype=torch.int32, device="cuda")
    choice = torch.zeros(rows, dtype=torch.int32, device="cuda")
    path = torch.zeros((R, gamma), dtype=torch.int32, device="cuda")

    def step():
        pool.plan(length, parent=parent)
        for i, cache in enumerate(caches):
            pool.append(cache, kv[i, :, :HEADS], kv[i, :, HEADS:])
            pool.attend(cache, q[i], gamma + 1, out[i], lse[i])
        pool.accept(tokens, choice, path, parent=parent)
        for cache in caches:
            pool.compact(cache, path)

    state = [pool.ctx, pool.held, pool.free_pages, pool.n_free, pool.block_table]
    state += [t for cache in caches for t in (cache.k, cache.v)]
    start = [t.clone() for t in state]
    results = state + [pool.row_start, pool.position, pool.slot, pool.anc, pool.accepted,
                       pool.bonus, pool.ctx_before, path, out, lse]

    def reset(seed):
        for t, was in zip(state, start):
            t.copy_(was)
        pool.ctx.sub_(i32([0, 40 * seed, 0]))
        kv.copy_(normal(kv.shape, 60 + seed))
        q.copy_(normal(q.shape, 70 + seed))
        g = torch.Generator(device="cuda")
        g.manual_seed(80 + seed)
        for t in (tokens, choice):
            t.copy_(torch.randint(0, 2, t.shape, generator=g, device="cuda"))
        out.zero_()
        lse.zero_()

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    accepted = []
    for seed in range(4):
        reset(seed)
        step()
        want = [t.clone() for t in results]
        reset(seed)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        raw = lambda t: t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t  # noqa: E731
        for a, b in zip(results, want):
            assert torch.equal(raw(a), raw(b))
        accepted += host(pool.accepted).tolist()
    assert len(set(accepted)) > 1 and dsp.dspark_device_status() == 0


@TYPES
def test_a_replay_beside_attends_of_the_stream_it_was_captured_on(fp8):
    pool, caches = long_contexts(2, fp8)
    pool.plan(i32([7, 7, 7]))
    qs = [normal((pool.n_rows, HEADS * GROUP, DIM), 95 + i) for i in range(2)]
    want = [torch.zeros_like(q) for q in qs]
    for cache, q, out in zip(caches, qs, want):
        pool.attend(cache, q, 8, out)
    stream, other = torch.cuda.Stream(), torch.cuda.Stream()
    held = torch.zeros_like(qs[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        pool.attend(caches[0], qs[0], 8, held)
    got = [[torch.zeros_like(q) for _ in range(20)] for q in qs]
    torch.cuda.synchronize()
    for k in range(20):
        with torch.cuda.stream(other):
            held.zero_()
            graph.replay()
            got[0][k].copy_(held)
        pool.attend(caches[1], qs[1], 8, got[1][k], stream=stream)
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(out, want[i]) for out in got[i])


@TYPES
def test_rounds_on_a_side_stream(fp8):
    # every call of several rounds on a stream that is named, none waited for
    def rounds(stream):
        pool, (cache,) = long_contexts(1, fp8)
        length, step = i32([7, 0, 3]), i32([5, 1, 2])
        kv = [normal((pool.n_rows, 2 * HEADS, DIM), 100 + i) for i in range(8)]
        q = [normal((pool.n_rows, HEADS * GROUP, DIM), 110 + i) for i in range(8)]
        outs = [torch.zeros_like(x) for x in q]
        seen = torch.zeros((8, 3), dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        for i in range(8):
            pool.plan(length, stream=stream)
            pool.append(cache, kv[i][:, :HEADS], kv[i][:, HEADS:], stream=stream)
            pool.attend(cache, q[i], 8, outs[i], stream=stream)
            pool.commit(step, stream=stream)
            with torch.cuda.stream(stream):
                seen[i].copy_(pool.ctx)
        torch.cuda.synchronize()
        return outs, seen

    want, ctx = rounds(None)
    assert ctx[:, 0].tolist() == list(range(2505, 2545, 5))
    got, ctx2 = rounds(torch.cuda.Stream())
    assert torch.equal(ctx, ctx2) and all(torch.equal(a, b) for a, b in zip(got, want))
