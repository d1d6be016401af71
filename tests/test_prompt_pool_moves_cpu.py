"""What PagePool's copies and moves hold before there is anything to copy or move, without a
GPU."""
import torch

from test_cache_pool_cpu import CACHE, calls  # noqa: F401
from test_prompt_pool_cpu import more, pool  # noqa: F401


def test_a_pool_that_was_never_squeezed_moves_nothing(more, monkeypatch):  # noqa: F811
    new = torch.empty
    # memory as an allocator gives it that was used before
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: new(*a, **kw).fill_(3))
    p = pool(shared=True)
    p.move(CACHE)
    assert more[-1].name == "dspark_kv_copy" and (more[-1].args[1] < 0).all()
    assert int(p.n_moves) == 0
