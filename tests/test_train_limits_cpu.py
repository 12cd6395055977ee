"""Extents that the descriptors' 32-bit fields do not hold are refused by the
binding instead of being cut off.  Runs without a GPU.
"""
import pytest
import torch

from backward_implicit_gemm_amd import binding as gb

WRAPS = 2 ** 32     # a multiple of what a field holds: cut off, 2^32 + 4 would be 4


@pytest.mark.parametrize("change", [dict(dim=WRAPS + 4), dict(vocab=WRAPS + 10), dict(tokens=WRAPS + 3), dict(rows=2 ** 64 + 2),
                                    dict(dim=2 ** 31), dict(vocab=2 ** 31)])
def test_embedding(change):
    with pytest.raises(ValueError, match="invalid embedding"):
        gb.Embedding(**dict(rows=2, tokens=3, vocab=10, dim=4, dtype=torch.float32, device="cpu") | change)


@pytest.mark.parametrize("shape,groups", [((WRAPS + 2, 8, 3, 4), 2), ((2, WRAPS + 8, 3, 4), 2), ((2, 8, WRAPS + 3, 4), 2),
                                          ((2, 8, 3, WRAPS + 4), 2), ((2, 2 ** 31, 1, 1), 2 ** 31)])
def test_group_norm(shape, groups):
    with pytest.raises(ValueError, match="invalid group norm"):
        gb.GroupNorm(shape, groups, "relu", torch.float32, device="cpu")
