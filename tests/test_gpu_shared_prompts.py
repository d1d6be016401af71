"""The example of forked prompts runs, in both types of cache, with short and long chunks, and
agrees with every continuation by itself wherever the choice is clear."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("chunk", [30, 100, 500])
def test_continuations(chunk, fp8):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import shared_prompts
    got = shared_prompts.main(["--check", "--chunk", str(chunk), "--tokens", "6"] + ["--fp8"] * fp8)
    assert len(got) == shared_prompts.PROMPTS * shared_prompts.SAMPLES
    assert all(len(t) in (4, 7) for t in got)
