"""Operands of a prompt's calls that lie on another device, without a GPU: stand-ins that say
where they are, and a library that only counts the calls that reach it."""
import pytest
import torch

import speculative_decoding_draft_02_gb300 as dsp

I32, BF16 = torch.int32, torch.bfloat16


class On:
    """A tensor that says it lies on the given GPU."""
    is_cuda = True

    def __init__(self, tensor, device=0):
        self.tensor, self.device_index = tensor, device

    def __getattr__(self, name):
        return getattr(self.tensor, name)

    def get_device(self):
        return self.device_index


class Library:
    def __init__(self):
        self.reached = []

    def __getattr__(self, name):
        def call(*args):
            self.reached.append(name)
            return 0
        return call


@pytest.fixture
def library(monkeypatch):
    got = Library()
    monkeypatch.setattr(dsp, "load_library", lambda: got)
    monkeypatch.setattr(dsp, "_device", lambda: 0)
    monkeypatch.setattr(dsp, "_stream", lambda stream: 0)
    return got


def zeros(*shape, dtype=I32, device=0):
    return On(torch.zeros(shape, dtype=dtype), device)


def cache(device=0):
    return dsp.KVCache(*(zeros(4, 16, 2, 64, dtype=BF16, device=device) for _ in range(2)))


def rotary(device=0, n=32):
    r = dsp.Rotary([0.5] * n, device="cpu")
    if device is not None:
        r.turns = On(r.turns, device)
    return r


def rope(rot, c=None, **kw):
    heads = [zeros(3, 2, 64, dtype=BF16) for _ in range(4)]
    a = dict(q=heads[0], k=heads[1], v=heads[2], position=zeros(3), slot=zeros(3, dtype=torch.int64),
             q_out=heads[3], q_weight=zeros(64, dtype=BF16), k_weight=zeros(64, dtype=BF16))
    a.update(kw)
    dsp.dspark_rope_append(c or cache(), rotary=rot, **a)


@pytest.mark.parametrize("device", [None, 1], ids=["host", "another_gpu"])
def test_a_rotation_of_another_device_is_refused(library, device):
    rope(rotary())
    assert library.reached == ["dspark_rope_append"]
    with pytest.raises(dsp.DSparkError, match="rotary"):
        rope(rotary(device))
    assert library.reached == ["dspark_rope_append"]
    rope(rotary(device, n=0))       # nothing turns, and no table is read
    assert len(library.reached) == 2
