"""The attention over more requests than a CTA has threads (384, or 512 beside an 8-bit
cache): a thread of the list's scan then has several, and finds its CTA's first among
them.  And over contexts of one, two and three tiles in turn, where the two sets of
softmax warps stand at the ends of different segments at once.  Held to the float64
oracle with the tolerances of test_gpu_cache, and to the same bits from call to call."""
import numpy as np
import pytest
import torch

from test_gpu_cache import attention_case, check_attention, run_attention, _lib  # noqa: F401

pytestmark = pytest.mark.gpu

TYPES = pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])


@TYPES
@pytest.mark.parametrize("R,tree,empty", [(384, False, 0.0), (385, True, 0.3), (512, True, 0.0),
                                          (513, False, 0.5), (1025, True, 0.4), (2000, False, 0.9)])
def test_many_requests(R, tree, empty, fp8):
    rng = np.random.default_rng(R)
    ctx = rng.integers(0, 300, R)
    ctx[rng.random(R) < 0.5] //= 20
    ns = rng.integers(1, 5, R)
    ns[rng.random(R) < empty] = 0
    ns[R // 3:R // 3 + 40 * (empty > 0)] = 0       # a run without rows, longer than a thread's share
    ns[-3:] = [2, 0, 0]
    c = attention_case([int(x) for x in ctx], [int(x) for x in ns], 2, 1, 64, 16, fp8=fp8,
                       tree=tree, seed=R)
    out, lse = run_attention(c)
    check_attention(c, out, lse)
    again, lse2 = run_attention(c)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@TYPES
@pytest.mark.parametrize("group,rows", [(1, 1), (4, 5), (8, 6), (16, 4)])
@pytest.mark.parametrize("tiles", [(1, 2), (1, 1, 2), (1, 2, 3), (1, 3, 2, 1, 4)], ids=str)
def test_items_of_few_tiles_in_turn(tiles, group, rows, fp8):
    # a set's part of an item may end while the other is at the end of the item before
    R = 200
    rng = np.random.default_rng(len(tiles))
    ctx = [128 * tiles[r % len(tiles)] - int(rng.integers(rows, 60)) for r in range(R)]
    c = attention_case(ctx, [rows] * R, 2 * group, 2, 64, 16, fp8=fp8, seed=group)
    out, lse = run_attention(c)
    for _ in range(10):
        again, lse2 = run_attention(c)
        assert torch.equal(out, again) and torch.equal(lse, lse2)
    few = {k: v[:12] if k in ("ctx", "ns", "table") else v for k, v in c.items()}
    few["row_start"] = c["row_start"][:13]
    few["q"] = c["q"][:12 * rows]
    pad = torch.full_like(out[:3], -77.0)
    check_attention(few, torch.cat([out[:12 * rows], pad]),
                    torch.cat([lse[:12 * rows], torch.full_like(lse[:3], -77.0)]))
