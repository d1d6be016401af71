"""Sizes of a prompt's calls that other tests leave out: rotation beside a single KV head at
many rows, and a pool's chunks of up to 64 rows, against the float64 oracle."""
import numpy as np
import pytest

from oracle import prompt as op
from test_gpu_cache import dsp, host, make_cache, i32, _lib  # noqa: F401
from test_gpu_prompt_pool import TYPES, caches_of, make_pool, rotary, step
from test_gpu_rope import compare, inv_freq, rows_case, run

pytestmark = pytest.mark.gpu


@TYPES
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rows,heads_q", [(1500, 1), (701, 5)])
def test_rotation_beside_one_kv_head(rows, heads_q, dim, fp8):
    rng = np.random.default_rng(rows + dim)
    n_pages = -(-rows // 16) + 1
    cache = make_cache(n_pages, 16, 1, dim, fp8, seed=rows)
    (q, k, v), weights = rows_case(rows, heads_q, 1, dim, rows + 1, std=3.0)
    position = rng.integers(0, 5000, rows)
    slot = rng.permutation(n_pages * 16)[:rows]
    position[[5, 60]], slot[[7, 8, rows - 1]] = -1, -1
    f = inv_freq(dim)
    ws = [host(w).astype(np.float64) for w in weights]
    ks, vs = (None if s is None else host(s).astype(np.float64) for s in (cache.k_scale, cache.v_scale))
    want_q, want_k, want_v = op.rope_append(
        host(q), host(k), host(v), position, slot, f, False, *ws, 1e-5, np.full(q.shape, -77.0),
        host(cache.k), host(cache.v), ks, vs)
    out = run(cache, q, k, v, position, slot, dsp.Rotary(f), weights, 1e-5)
    compare(host(out), want_q, 2.0 ** -8)
    np.testing.assert_array_equal(host(cache.v), want_v)
    if fp8:
        compare(host(cache.k), np.clip(want_k, -448, 448), 2.0 ** -4, 2.0 ** -10)
    else:
        compare(host(cache.k), want_k, 2.0 ** -8)


@TYPES
def test_a_pools_chunks_of_few_rows(fp8):
    pool = make_pool(R=4)
    caches, rot = caches_of(pool, fp8), rotary()
    pool.ctx.zero_()
    for i, ns in enumerate(([200, 64, 33, 1], [64, 40, 33, 9], [0, 33, 1, 64])):
        step(pool, caches, ns, rot, i + 1)
        pool.commit(i32(ns))
    assert dsp.dspark_device_status() == 0
