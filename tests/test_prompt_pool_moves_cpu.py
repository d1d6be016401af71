"""What PagePool's copies and moves hold before there is anything to copy or move, without a
GPU."""
import pytest
import torch

import speculative_decoding_draft_02_gb300 as dsp

from test_cache_pool_cpu import CACHE, calls  # noqa: F401
from test_prompt_pool_cpu import I32, more, pool  # noqa: F401


def test_a_pool_that_was_never_squeezed_moves_nothing(more, monkeypatch):  # noqa: F811
    new = torch.empty
    # memory as an allocator gives it that was used before
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: new(*a, **kw).fill_(3))
    p = pool(shared=True)
    p.move(CACHE)
    assert more[-1].name == "dspark_kv_copy" and (more[-1].args[1] < 0).all()
    assert int(p.n_moves) == 0


def test_a_fork_that_was_refused_leaves_the_last_ones_copies(more, monkeypatch):  # noqa: F811
    p = pool(shared=True)
    three, two = torch.zeros(3, dtype=I32), torch.zeros(2, dtype=I32)

    def refused(*args):
        raise dsp.DSparkError("refused")

    accepted = dsp.dspark_kv_fork
    for ready, copies in ((False, 0), (True, 3)):
        if ready:
            monkeypatch.setattr(dsp, "dspark_kv_fork", accepted)
            p.fork(three, three)
        monkeypatch.setattr(dsp, "dspark_kv_fork", refused)
        with pytest.raises(dsp.DSparkError, match="refused"):
            p.fork(two, two)
        p.copy(CACHE)
        assert [t.numel() for t in more[-1].args[1:4]] == [copies] * 3


def test_a_fork_releases_first(more):  # noqa: F811
    p = pool(shared=True)
    one = torch.zeros(1, dtype=I32)
    p.fork(one, one, stream="s")
    assert [c.name for c in more] == ["dspark_kv_release", "dspark_kv_fork"]
    assert all(c.args[-1] == "s" for c in more)
