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
