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


def calls():
    """Each call of a prompt's way as (function, tensor arguments by name, the others)."""
    heads = [zeros(3, 2, 64, dtype=BF16) for _ in range(4)]
    bf16 = dict(dtype=BF16)
    R, pages, table = 2, 6, lambda: zeros(2, 3)  # noqa: E731
    tables = dict(ctx=zeros(R), held=zeros(R), n_free=zeros(1), free_pages=zeros(pages),
                  block_table=table(), refs=zeros(pages))
    return [
        (dsp.dspark_rope_append,
         dict(q=heads[0], k=heads[1], v=heads[2], q_out=heads[3], q_weight=zeros(64, **bf16),
              k_weight=zeros(64, **bf16), position=zeros(3), slot=zeros(3, dtype=torch.int64)),
         dict(rotary=rotary())),
        (dsp.dspark_chunk_attention,
         dict(q=heads[0], out=heads[3], ctx=zeros(R), row_start=zeros(R + 1), block_table=table(),
              lse=zeros(3, 2, dtype=torch.float32), workspace=zeros(512, dtype=torch.uint8)),
         dict(max_rows=3, scale=0.1)),
        (dsp.dspark_kv_fork, dict(source=zeros(1), target=zeros(1), copy_from=zeros(1),
                                  copy_to=zeros(1), copy_tokens=zeros(1), **tables),
         dict(page_size=16)),
        (dsp.dspark_kv_release, dict(tables), {}),
        (dsp.dspark_kv_squeeze,
         dict({k: v for k, v in tables.items() if k != "ctx"}, free_pages_out=zeros(pages),
              block_table_out=table(), refs_out=zeros(pages), new_page=zeros(pages),
              move_from=zeros(3), move_to=zeros(3), n_moves=zeros(1)), {}),
        (dsp.dspark_kv_copy, dict(copy_from=zeros(2), copy_to=zeros(2), copy_tokens=zeros(2)), {}),
    ]


@pytest.mark.parametrize("i", range(6))
def test_every_tensor_of_another_device_is_refused(library, i):
    call, tensors, rest = calls()[i]
    if "kv_" not in call.__name__ or call is dsp.dspark_kv_copy:
        rest["cache"] = cache()
    call(**tensors, **rest)
    assert library.reached == [call.__name__]
    for name, t in tensors.items():
        for where in (1, -1):
            away = On(t.tensor, where)
            away.is_cuda = where >= 0
            with pytest.raises(dsp.DSparkError):
                call(**{**tensors, name: away}, **rest)
    if "cache" in rest:
        with pytest.raises(dsp.DSparkError, match="cache"):
            call(**tensors, **{**rest, "cache": cache(1)})
    for t in tensors.values():      # all together on a device that is not the current one
        t.device_index = 1
    if "cache" in rest:
        rest["cache"] = cache(1)
    if "rotary" in rest:
        rest["rotary"] = rotary(1)
    with pytest.raises(dsp.DSparkError, match="current"):
        call(**tensors, **rest)
    assert library.reached == [call.__name__]


def test_a_cache_lies_on_one_device():
    k, v = (torch.zeros((4, 16, 2, 64), dtype=torch.float8_e4m3fn) for _ in range(2))
    s = torch.ones(2)
    dsp.KVCache(On(k), On(v), On(s), On(s))
    for bad in ((On(k), On(v, 1)), (On(k), On(v), On(s, 1), On(s)), (On(k), On(v), On(s), On(s, 1))):
        with pytest.raises(dsp.DSparkError):
            dsp.KVCache(*bad)
