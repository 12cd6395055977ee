"""A scale that is not finite is refused: infinity times the zero sum of a table row
without a token would be NaN, and the two forms of the gradient would differ there.
Runs without a GPU.
"""
import ctypes

import pytest
import torch

from backward_implicit_gemm_amd import binding as gb

FAKE = 0x10000     # never dereferenced: every call below fails validation


@pytest.mark.parametrize("scale", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("V", [10, 100000], ids=["small table", "sorted"])
def test_refused(V, scale):
    d = gb.gc_embed_desc(4, 3, V, 8, gb.GC_I32, 24, 3)
    assert gb.lib().gc_embed_fwd(FAKE, FAKE, FAKE, ctypes.byref(d), scale, 0, None) == gb.GC_ERR_INVALID_ARG
    assert gb.lib().gc_embed_bwd(FAKE, FAKE, FAKE, FAKE, 1 << 40, ctypes.byref(d), scale, 0, None) == gb.GC_ERR_INVALID_ARG
    with pytest.raises(ValueError, match="finite"):
        gb.Embedding(4, 3, V, 8, torch.float32, scale, device="cpu")


def test_refused_past_the_range_of_fp32():
    with pytest.raises(ValueError, match="finite"):
        gb.Embedding(4, 3, 10, 8, torch.float32, 1e39, device="cpu")
