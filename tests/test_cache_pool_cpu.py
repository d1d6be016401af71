"""PagePool's own dealings (which masks, which scratch, which stream go into a call),
without a GPU: the entry points are replaced by recorders."""
import contextlib
from types import SimpleNamespace

import pytest
import torch

import speculative_decoding_draft_02_gb300 as dsp


class Scratch:
    def record_stream(self, stream):
        pass


@pytest.fixture
def calls(monkeypatch):
    """The arguments of every entry point that the pool calls, by name."""
    got = []

    def record(name, result=None):
        def call(*args, **kw):
            got.append(SimpleNamespace(name=name, args=args, kw=kw))
            return result
        monkeypatch.setattr(dsp, name, call)

    record("dspark_kv_plan")
    record("dspark_kv_append")
    record("dspark_tree_attention")
    record("dspark_tree_attention_workspace_bytes", 512)
    # the streams here are stand-ins, and no current one exists
    monkeypatch.setattr(dsp, "_stream", lambda s: 0 if s is None else s.cuda_stream)
    monkeypatch.setattr(dsp, "workspace", lambda n, device: Scratch())
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return got


def make_pool():
    return dsp.PagePool(2, 8, 16, 64, 32, device="cpu")


CACHE = SimpleNamespace(dim=64)
Q = torch.zeros((32, 4, 64), dtype=torch.bfloat16)


def masks_of(pool, calls):
    pool.attend(CACHE, Q, 8, Q.clone())
    call = calls[-1]
    assert call.name == "dspark_tree_attention"
    return call.args[4]


def test_a_prompts_rows_are_attended_as_chains(calls):
    pool = make_pool()
    two = torch.full((2,), 2, dtype=torch.int32)
    pool.plan(two, extra=0)
    assert calls[-1].args[14] is None     # no masks are written for prompts
    assert masks_of(pool, calls) is None  # so none may be read: chains
    pool.plan(two)
    assert calls[-1].args[14] is pool.anc and masks_of(pool, calls) is pool.anc
    pool.plan(two, extra=0)
    assert masks_of(pool, calls) is None


def scratch_of(pool, calls, **kw):
    pool.attend(CACHE, Q, 8, Q.clone(), **kw)
    return calls[-1].args[10]


def test_streams_do_not_share_scratch(calls, monkeypatch):
    # an attention's pieces lie in its scratch until its join has read them
    pool = make_pool()
    one, two = SimpleNamespace(cuda_stream=11), SimpleNamespace(cuda_stream=12)
    at = [scratch_of(pool, calls, stream=s) for s in (None, one, two)]
    assert len(set(at)) == 3
    # kept for the next call there
    assert all(scratch_of(pool, calls, stream=s) is t for s, t in zip((None, one, two), at))
    # the current stream's, where none is named
    monkeypatch.setattr(dsp, "_stream", lambda s: 12 if s is None else s.cuda_stream)
    assert scratch_of(pool, calls) is at[2]
    # a graph may be replayed on any stream: its scratch is its own
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    held = [scratch_of(pool, calls, stream=s) for s in (one, one, None)]
    assert not set(held) & set(at)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    assert scratch_of(pool, calls, stream=one) is at[1]


@pytest.mark.parametrize("rows", [torch.tensor([3, 9], dtype=torch.int32), torch.tensor([3, 9]), 3],
                         ids=["int32", "int64", "number"])
def test_commit_goes_on_the_stream_that_is_named(calls, monkeypatch, rows):
    # what it changes is read by the kernels of that stream
    pool = make_pool()
    pool.ctx.copy_(torch.tensor([7, -1]))
    inside = []

    class On(contextlib.AbstractContextManager):
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            inside.append(self.stream)
            self.before = pool.ctx.clone()

        def __exit__(self, *_):
            inside.append(not torch.equal(self.before, pool.ctx))

    monkeypatch.setattr(torch.cuda, "stream", On)
    s = SimpleNamespace(cuda_stream=5)
    pool.commit(rows, stream=s)
    assert inside == [s, True]              # the change was made within
    assert pool.ctx.tolist() == [10, -1] and pool.ctx.dtype is torch.int32
    pool.commit(rows)
    assert inside == [s, True, None, True] and pool.ctx.tolist() == [13, -1]
