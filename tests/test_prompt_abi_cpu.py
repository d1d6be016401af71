"""The entry points of a prompt's way into the cache, and their binding, without a GPU:
every refusal comes before anything is launched, and none needs a device."""
import ctypes
import math

import numpy as np
import pytest
import torch

import speculative_decoding_draft_02_gb300 as dsp
from speculative_decoding_draft_02_gb300 import build as dsp_build
from test_cache_abi_cpu import cache

FAKE = ctypes.c_void_p(4096)


@pytest.fixture(scope="module")
def lib():
    dsp_build.build()
    return dsp.load_library()


BAD_CACHES = [dict(k=None), dict(v=None), dict(k=4100), dict(dim=96), dict(heads=0),
              dict(page_size=48), dict(n_pages=0), dict(type=2), dict(token_stride=60),
              dict(head_stride=-64), dict(page_stride=1 << 41), dict(type=1, head_stride=72)]


def rope(lib, c=None, rows=1, heads_q=4, q=FAKE, q_row=256, q_head=64, k=FAKE, v=FAKE, kv_row=128,
         kv_head=64, qw=FAKE, kw=FAKE, eps=1e-6, turns=4096, dims=64, style=0, rotary=True,
         position=FAKE, slot=FAKE, out=FAKE, out_row=256, out_head=64):
    r = ctypes.byref(dsp.RopeStruct(turns, dims, style)) if rotary else None
    return lib.dspark_rope_append(cache() if c is None else c, rows, heads_q, q, q_row, q_head, k, v,
                                  kv_row, kv_head, qw, kw, eps, r, position, slot, out, out_row,
                                  out_head, None)


@pytest.mark.parametrize("kw", BAD_CACHES, ids=str)
def test_caches_that_are_refused(lib, kw):
    c = cache(**kw)
    assert rope(lib, c) == 1
    assert lib.dspark_chunk_attention_workspace_bytes(c, 4, 8, 100) == 0
    assert lib.dspark_chunk_attention(c, 1, 8, 100, 100, 1, FAKE, 512, 64, FAKE, FAKE, FAKE, 0.1, FAKE,
                                      512, 64, None, FAKE, 1 << 40, None) == 1
    assert lib.dspark_kv_copy(c, 1, FAKE, FAKE, None, None) == 1


ODD = ctypes.c_void_p(4104)


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(heads_q=0), dict(heads_q=-4), dict(heads_q=65536), dict(q=None), dict(k=None),
    dict(v=None), dict(position=None), dict(slot=None), dict(out=None), dict(q=ODD), dict(k=ODD),
    dict(v=ODD), dict(out=ODD), dict(qw=ODD), dict(kw=ODD), dict(q_row=0), dict(q_head=60),
    dict(kv_row=-64), dict(kv_head=4), dict(out_row=1 << 39), dict(out_head=12), dict(eps=-1e-6),
    dict(eps=math.nan), dict(rotary=False), dict(turns=None), dict(turns=4100), dict(dims=-16),
    dict(dims=80), dict(dims=24), dict(style=2), dict(style=-1)], ids=str)
def test_rotations_that_are_refused(lib, kw):
    assert rope(lib, **kw) == 1
    assert rope(lib, **{"rows": 0, **{k: v for k, v in kw.items() if k in ("dims", "style")}}) in (0, 1)


def test_nothing_to_do(lib):
    assert rope(lib, rows=0) == 0
    assert rope(lib, rows=0, q=None, k=None, v=None, position=None, slot=None, out=None) == 0
    assert lib.dspark_kv_copy(cache(), 0, None, None, None, None) == 0
    assert lib.dspark_kv_fork(0, None, None, 4, 16, 8, 2, *[None] * 9, None) == 0
    assert lib.dspark_chunk_attention(cache(), 1, 8, 100, 0, 1, None, 0, 0, None, None, None, 0.1, None,
                                      0, 0, None, None, 0, None) == 0


def chunk(lib, R=1, heads_q=8, max_rows=100, rows=100, pages=1, q=FAKE, q_row=512, q_head=64, ctx=FAKE,
          start=FAKE, table=FAKE, out=FAKE, out_row=512, out_head=64, ws=FAKE, size=1 << 40):
    return lib.dspark_chunk_attention(cache(), R, heads_q, max_rows, rows, pages, q, q_row, q_head, ctx,
                                      start, table, 0.1, out, out_row, out_head, None, ws, size, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(R=0), 1), (dict(heads_q=7), 1), (dict(heads_q=0), 1), (dict(heads_q=2 * 65), 1),
    (dict(max_rows=0), 1), (dict(max_rows=-5), 1), (dict(rows=-1), 1), (dict(pages=0), 1),
    (dict(q=None), 1), (dict(q=ODD), 1), (dict(q_row=4), 1), (dict(q_head=0), 1),
    (dict(q_row=1 << 39), 1), (dict(ctx=None), 1), (dict(start=None), 1), (dict(table=None), 1),
    (dict(out=None), 1), (dict(out=ODD), 1), (dict(out_row=-8), 1), (dict(out_head=68), 1),
    (dict(out_row=1 << 39), 1), (dict(ws=None), 4), (dict(ws=ODD), 4), (dict(size=100), 4)], ids=str)
def test_attentions_that_are_refused(lib, kw, rc):
    kw = {k: ctypes.c_void_p(4352) if v is ODD and k == "ws" else v for k, v in kw.items()}
    if kw.get("ws") is not None:
        kw["ws"] = ctypes.c_void_p(4112)
    assert chunk(lib, **kw) == rc
    if max(kw.get("max_rows", 100), 0) > 0:
        assert chunk(lib, **{**kw, "max_rows": 5}) == rc  # as the tree attention's call


def test_workspace_sizes(lib):
    size = lib.dspark_chunk_attention_workspace_bytes
    for R, heads_q, rows in ((0, 8, 6), (4, 0, 6), (4, 7, 6), (4, 8, 0), (4, 2 * 65, 100)):
        assert size(cache(), R, heads_q, rows) == 0, (R, heads_q, rows)
    assert size(None, 4, 8, 100) == 0


def test_tables_that_are_refused(lib):
    def fork(n=1, R=4, ps=16, pages=8, most=2, null=None):
        ptr = [FAKE] * 11
        if null is not None:
            ptr[null] = None
        return lib.dspark_kv_fork(n, *ptr[:2], R, ps, pages, most, *ptr[2:], None)

    for kw in (dict(n=-1), dict(R=0), dict(ps=24), dict(ps=8), dict(ps=512), dict(pages=0), dict(most=0)):
        assert fork(**kw) == 1, kw
    for i in range(11):
        assert fork(null=i) == 1, i
    assert fork(n=5) == 8 and fork(R=16385) == 8

    def release(R=4, pages=8, most=2, null=None):
        ptr = [FAKE] * 6
        if null is not None:
            ptr[null] = None
        return lib.dspark_kv_release(R, pages, most, *ptr, None)

    for kw in (dict(R=0), dict(R=-1), dict(pages=0), dict(most=0)):
        assert release(**kw) == 1, kw
    for i in range(6):
        assert release(null=i) == 1, i
    assert release(R=16385) == 8

    def squeeze(R=4, pages=8, most=2, null=None):
        ptr = [FAKE] * 12
        if null is not None:
            ptr[null] = None
        return lib.dspark_kv_squeeze(R, pages, most, *ptr, None)

    for kw in (dict(R=0), dict(pages=1), dict(pages=-1), dict(most=0)):
        assert squeeze(**kw) == 1, kw
    for i in range(12):
        assert squeeze(null=i) == 1, i
    assert squeeze(R=16385) == 8
    assert lib.dspark_kv_copy(cache(), -1, FAKE, FAKE, None, None) == 1
    assert lib.dspark_kv_copy(cache(), 1, None, FAKE, None, None) == 1
    assert lib.dspark_kv_copy(cache(), 1, FAKE, None, None, None) == 1


def test_a_rotarys_turns():
    f = [0.0, 2 * math.pi / 4, 2 * math.pi, 2 * math.pi * 1.25, -2 * math.pi / 4, 1.0, 1e-6, math.pi]
    r = dsp.Rotary(f, device="cpu")
    turns = [int(x) % 2 ** 64 for x in r.turns]
    assert turns[:5] == [0, 2 ** 62, 0, 2 ** 62, 3 * 2 ** 62] and turns[7] == 2 ** 63
    for x, t in zip(f[5:7], turns[5:7]):
        assert abs(t - x / (2 * math.pi) * 2 ** 64) <= 2 ** 11
    assert r.dims == 16 and r.struct.style == dsp.ROPE_HALVES
    assert dsp.Rotary(torch.zeros(24, dtype=torch.float64), pairs=True, device="cpu").struct.style == 1
    assert dsp.Rotary([], device="cpu").dims == 0
    for bad in ([0.5] * 7, [math.nan] * 8, [math.inf] * 8, np.zeros((2, 8))):
        with pytest.raises(dsp.DSparkError):
            dsp.Rotary(bad, device="cpu")


def test_the_binding_wants_gpu_tensors():
    i = torch.zeros(2, dtype=torch.int32)
    table = torch.zeros((2, 1), dtype=torch.int32)
    with pytest.raises(dsp.DSparkError):
        dsp.dspark_kv_fork(i, i, 16, i, i, i[:1], i, table, i, i, i, i)
    with pytest.raises(dsp.DSparkError):
        dsp.dspark_kv_release(i, i, i[:1], i, table, i)
    with pytest.raises(dsp.DSparkError):
        dsp.dspark_kv_squeeze(i, i[:1], i, table, i, i, table, i, i, i[:1], i[:1], i[:1])


def test_a_pool_that_shares_nothing_refuses_to():
    pool = dsp.PagePool(2, 8, 16, 64, 32, device="cpu")
    i = torch.zeros(1, dtype=torch.int32)
    for call in (lambda: pool.fork(i, i), lambda: pool.copy(None), pool.release, pool.squeeze,
                 lambda: pool.move(None)):
        with pytest.raises(dsp.DSparkError, match="shared"):
            call()
    pool = dsp.PagePool(2, 8, 16, 64, 32, device="cpu", shared=True)
    with pytest.raises(dsp.DSparkError, match="places"):
        pool.fork(torch.zeros(3, dtype=torch.int32), torch.zeros(3, dtype=torch.int32))


def test_tensors_of_another_device_are_refused(monkeypatch):
    from types import SimpleNamespace
    monkeypatch.setattr(dsp, "_device", lambda: 1)
    monkeypatch.setattr(dsp, "_stream", lambda stream: 77)
    with pytest.raises(dsp.DSparkError, match="device 0"):
        dsp._stream_on("call", SimpleNamespace(get_device=lambda: 0), None)
    assert dsp._stream_on("call", SimpleNamespace(get_device=lambda: 1), None) == 77
