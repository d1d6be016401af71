"""Attention of chunks where the list of work or a tile's end is unusual, against the float64
oracle, with the tolerances of test_gpu_chunk."""
import math

import numpy as np
import pytest
import torch

from test_gpu_cache import dsp, host, i32, _lib  # noqa: F401
from test_gpu_chunk import case, check, run

pytestmark = pytest.mark.gpu

TYPES = pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])


@TYPES
@pytest.mark.parametrize("dim", [64, 128])
def test_rows_behind_the_end_of_their_table(dim, fp8):
    # a table that ends inside a tile, and rows whose own positions lie past it: they see the
    # table's tokens, and nothing of what an earlier call left in shared memory
    left = case([60000], [65], 2, 1, dim, 64, fp8=fp8, seed=1, poison=False)
    left["cache"].v.copy_(torch.full_like(left["cache"].v, math.nan, dtype=torch.float32).to(
        left["cache"].v.dtype))
    for ctx, pages in ((100, 10), (700, 10), (0, 3)):
        c = case([ctx, 30], [1000, 70], 4, 2, dim, 16, fp8=fp8, seed=ctx + dim)
        c["table"] = np.ascontiguousarray(c["table"][:, :pages])
        run(left)
        out, lse = run(c)
        assert dsp.dspark_device_status() == 6
        check(c, out, lse)


LISTS = {
    # one item cut into some 75 pieces: a join's second round of 32 CTAs, and its third
    "many_pieces": ([20000], [100], 4, 1, 64, 64),
    # a single row over a long context beside a chunk, and beside nothing
    "one_row_beside_a_chunk": ([30000, 0], [1, 400], 8, 2, 128, 64),
    "one_row_of_64_heads": ([9000], [1], 64, 1, 128, 32),
}


@TYPES
@pytest.mark.parametrize("name", LISTS)
def test_long_lists(name, fp8):
    c = case(*LISTS[name], fp8=fp8, seed=len(name), poison=False)
    out, lse = run(c)
    check(c, out, lse)
    again, lse2 = run(c)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@TYPES
@pytest.mark.parametrize("R", [385, 513, 1100])
def test_more_requests_than_threads(R, fp8):
    # a thread counts several requests, and finds a cut among its own
    rng = np.random.default_rng(R)
    ns = rng.integers(0, 4, R)
    ns[rng.random(R) < 0.02] = 130
    ns[rng.random(R) < 0.2] = 0
    ctx = rng.integers(0, 200, R)
    c = case(ctx.tolist(), ns.tolist(), 2, 1, 64, 16, fp8=fp8, seed=R)
    out, lse = run(c, max_rows=130)
    check(c, out, lse)


@TYPES
def test_a_list_whose_cost_passes_32_bits(fp8):
    # contexts near 2^31 over a short table: counted whole, attended as far as the table goes
    c = case([40, 0, 300, 0, 0], [130, 3, 70, 200, 1], 16, 8, 64, 16, fp8=fp8, seed=1, poison=False)
    rng = np.random.default_rng(2)
    for r, far in ((1, 2 ** 31 - 100), (4, 2 ** 31 - 1)):
        c["ctx"][r] = far
        c["table"][r] = rng.integers(0, c["cache"].n_pages, c["table"].shape[1])
    out, lse = run(c)
    assert dsp.dspark_device_status() == 6
    check(c, out, lse)


@pytest.mark.parametrize("ahead", [1, 31, 33])
def test_large_values_behind_a_reference_that_is_kept(ahead):
    # tiles whose scores pass the first one's by so many octaves, and V near the 2^64 up to which
    # nothing overflows: within 32 octaves the weights grow instead of the reference
    c = case([0, 700], [400, 150], 2, 1, 128, 16, seed=4)
    k, table = c["cache"].k, c["table"]
    c["scale"] = 0.125
    c["q"].zero_()
    c["q"][:, :, 0] = 8.0
    raw = k.float()
    for r, total in ((0, 400), (1, 850)):
        for p in range(total):
            raw[table[r, p // 16], p % 16, 0, 0] = 0.0 if p < 128 else ahead * math.log(2)
    k.copy_(raw.to(k.dtype))
    v = c["cache"].v
    v.copy_((v.float().clamp(-3.9, 3.9) * 2.0 ** 62).to(v.dtype))
    out, lse = run(c)
    assert np.isfinite(host(out[:550])).all()
    check(c, out, lse)
