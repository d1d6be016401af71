"""PagePool on the GPU: a prompt's rows after a tree's.  The attention is held to the
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
