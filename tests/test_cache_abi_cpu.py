"""The paged-cache entry points and their binding without a GPU: every refusal comes
before anything is launched, and none needs a device."""
import ctypes

import pytest
import torch

import speculative_decoding_draft_02_gb300 as dsp
from speculative_decoding_draft_02_gb300 import build as dsp_build

FAKE = ctypes.c_void_p(4096)


@pytest.fixture(scope="module")
def lib():
    dsp_build.build()
    return dsp.load_library()


def cache(**kw):
    f = dict(k=4096, v=8192, k_scale=None, v_scale=None, page_stride=16 * 2 * 64, token_stride=128,
             head_stride=64, n_pages=4, page_size=16, heads=2, dim=64, type=0)
    return ctypes.byref(dsp.KVCacheStruct(**{**f, **kw}))


@pytest.mark.parametrize("kw", [
    dict(k=None), dict(v=None), dict(k=4100), dict(dim=0), dict(dim=96), dict(dim=256),
    dict(heads=0), dict(heads=-1), dict(page_size=0), dict(page_size=48), dict(page_size=8),
    dict(page_size=512), dict(n_pages=0), dict(n_pages=-3), dict(type=2), dict(type=-1),
    dict(token_stride=60), dict(token_stride=0), dict(head_stride=-64), dict(page_stride=4),
    dict(page_stride=1 << 41), dict(type=1, head_stride=72)], ids=str)
def test_caches_that_are_refused(lib, kw):
    assert lib.dspark_tree_attention_workspace_bytes(cache(**kw), 4, 8, 6) == 0
    assert lib.dspark_kv_append(cache(**kw), 1, FAKE, FAKE, 128, 64, FAKE, None) == 1
    assert lib.dspark_kv_compact(cache(**kw), 1, 5, 2, FAKE, FAKE, FAKE, FAKE, None) == 1
    assert lib.dspark_tree_attention(cache(**kw), 1, 8, 1, 1, 1, FAKE, 512, 64, FAKE, FAKE, None,
                                     FAKE, 0.1, FAKE, 512, 64, None, FAKE, 1 << 40, None) == 1


def test_sizes_that_are_refused(lib):
    size = lib.dspark_tree_attention_workspace_bytes
    for R, heads_q, nodes in ((0, 8, 6), (-1, 8, 6), (4, 0, 6), (4, 7, 6), (4, 1, 6), (4, 8, 0),
                              (4, 8, 65), (4, 2 * 65, 6)):
        assert size(cache(), R, heads_q, nodes) == 0, (R, heads_q, nodes)
    assert size(None, 4, 8, 6) == 0


def test_null_and_negative_arguments(lib):
    def plan(R=1, gamma=5, extra=1, rows=10, ps=16, pages=4, most=2, null=None):
        ptr = [FAKE] * 13
        if null is not None:
            ptr[null] = None
        return lib.dspark_kv_plan(R, gamma, extra, rows, ps, pages, most, *ptr, None)

    for kw in (dict(R=0), dict(R=-1), dict(gamma=-1), dict(gamma=64), dict(extra=-1), dict(extra=2),
               dict(rows=-1), dict(ps=24), dict(pages=-1), dict(most=0)):
        assert plan(**kw) == 1, kw
    for i in (0, 1, 3, 4, 5, 6, 7, 8, 9, 10, 11):  # all but the parents and the masks
        assert plan(null=i) == 1, i
    for i in range(9):
        if i == 1:                                 # chains
            continue
        ptr = [FAKE] * 9
        ptr[i] = None
        assert lib.dspark_tree_accept(1, 5, 6, *ptr, None) == 1, i
    for R, gamma, rows in ((0, 5, 6), (1, 64, 6), (1, -1, 6), (1, 5, -1)):
        assert lib.dspark_tree_accept(R, gamma, rows, *[FAKE] * 9, None) == 1
    for i in range(4):
        ptr = [FAKE] * 4
        ptr[i] = None
        assert lib.dspark_kv_compact(cache(), 1, 5, 2, *ptr, None) == 1
    assert lib.dspark_kv_append(cache(), -1, FAKE, FAKE, 128, 64, FAKE, None) == 1
    assert lib.dspark_kv_append(cache(), 0, None, None, 128, 64, None, None) == 0  # nothing to do


def test_the_binding_wants_gpu_tensors():
    k = torch.zeros((2, 16, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(dsp.DSparkError):
        dsp.KVCache(k, k)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(dsp.DSparkError):
        dsp.dspark_tree_accept(torch.zeros(2, dtype=torch.int32), None,
                               torch.zeros((1, 5), dtype=torch.int32), i, i, i, i,
                               torch.zeros((1, 5), dtype=torch.int32), i, stream=None)
    with pytest.raises(dsp.DSparkError):
        dsp.dspark_kv_plan(i, i, 1, None, 16, i, i, i, torch.zeros((1, 2), dtype=torch.int32), i, i,
                           torch.zeros(2, dtype=torch.int32), i, i.long())
