"""The paged-cache operators run together: the example's rounds emit what plain decoding
with the same target emits, with chains and with trees, and take several tokens a round."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import paged_round
    return paged_round


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("tree", [False, True], ids=["chain", "tree"])
def test_rounds_emit_the_targets_own_tokens(example, tree, fp8):
    args = ["--check", "--rounds", "6"] + ["--tree"] * tree + ["--fp8"] * fp8
    emitted = example.main(args)
    assert sum(map(len, emitted)) > 6 * example.R * 1.3
