"""PagePool's part in a prompt's way into the cache, without a GPU: which calls it makes, in
what order, with which of its tensors."""
from types import SimpleNamespace

import pytest
import torch

import speculative_decoding_draft_02_gb300 as dsp
from test_cache_pool_cpu import CACHE, Q, calls  # noqa: F401

I32 = torch.int32


@pytest.fixture
def more(calls, monkeypatch):  # noqa: F811
    def record(name, result=None):
        def call(*args, **kw):
            calls.append(SimpleNamespace(name=name, args=args, kw=kw))
            return result
        monkeypatch.setattr(dsp, name, call)

    record("dspark_chunk_attention")
    record("dspark_chunk_attention_workspace_bytes", 512)
    for name in ("rope_append", "kv_fork", "kv_release", "kv_squeeze", "kv_copy"):
        record("dspark_" + name)
    return calls


def pool(**kw):
    return dsp.PagePool(4, 8, 16, 64, 32, device="cpu", **kw)


def names(calls):  # noqa: F811
    got = [c.name for c in calls]
    calls.clear()
    return got


def test_prompts_of_many_rows_are_chunks(more):
    p, n = pool(), torch.full((4,), 2, dtype=I32)
    p.plan(n, extra=0)
    p.attend(CACHE, Q, 65, Q.clone())
    call = more[-1]
    assert call.name == "dspark_chunk_attention" and call.args[2] is p.ctx and call.args[5] == 65
    assert call.args[6] == 64 ** -0.5
    p.attend(CACHE, Q, 64, Q.clone())
    assert more[-1].name == "dspark_tree_attention" and more[-1].args[4] is None
    p.plan(n)                                # a round's rows are trees, however many are allowed
    p.attend(CACHE, Q, 65, Q.clone())
    assert more[-1].name == "dspark_tree_attention" and more[-1].args[4] is p.anc


def test_rotation_takes_the_planned_rows(more):
    p = pool()
    p.rope_append(CACHE, 1, 2, 3, 4, 5)
    assert more[-1].args[4] is p.position and more[-1].args[5] is p.slot


def test_a_shared_pool_releases_before_it_plans(more):
    n = torch.full((4,), 2, dtype=I32)
    p = pool()
    p.plan(n)
    assert names(more) == ["dspark_kv_plan"]
    p = pool(shared=True)
    p.plan(n)
    assert names(more) == ["dspark_kv_release", "dspark_kv_plan"]
    p.squeeze()
    assert names(more) == ["dspark_kv_release", "dspark_kv_squeeze"]


def test_copies_are_the_last_forks(more):
    p = pool(shared=True)
    p.copy(CACHE)
    assert more[-1].name == "dspark_kv_copy" and more[-1].args[1].numel() == 0
    i = torch.zeros(3, dtype=I32)
    p.fork(i, i)
    fork = more[-1].args
    p.copy(CACHE)
    got = more[-1].args[1:4]
    assert all(a is b and a.numel() == 3 for a, b in zip(fork[-4:-1], got))
    p.squeeze()
    squeeze = more[-1].args
    assert squeeze[2] is squeeze[5] is p.free_pages and squeeze[3] is squeeze[6] is p.block_table
    p.move(CACHE)
    assert more[-1].args[1] is p.move_from and more[-1].args[2] is p.move_to and more[-1].args[3] is None
