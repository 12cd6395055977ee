"""GPU: group norm of data with a few values far from all others, against the
definition in 64 bits.

One value of 10^3 to 10^6 deviations carries a group's sum of squares; it stands where
a thread of the kernels for large groups begins a block of its sums, or anywhere.  The
statistics have to stay within the bounds of train_ref, which hold for any data: they
count the additions a value goes through and nothing that cancels.
"""
import pytest
import torch

import train_ref as ref
from backward_implicit_gemm_amd import binding as gb

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5


def setup_module():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    gb.lib()


SHAPES = [
    ((8, 512, 64, 64), 16, "nchw"),      # planes in one piece
    ((64, 64, 128, 128), 8, "nchw"),
    ((2, 4, 300, 300), 2, "nchw"),       # and in several
    ((8, 512, 64, 64), 16, "nhwc"),
    ((4, 32, 150, 150), 2, "nhwc"),
    ((64, 128, 3, 4), 8, "nchw"),        # resident
    ((64, 128, 3, 4), 8, "nhwc"),
]


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("spike", [1e3, 3e4, 1e6])
@pytest.mark.parametrize("place", ["first", "anywhere", "first rows"])
@pytest.mark.parametrize("shape,G,layout", SHAPES, ids=[f"{'x'.join(map(str, s))}-{g}-{l}" for s, g, l in SHAPES])
def test_statistics_of_groups_with_outliers(shape, G, layout, place, spike, dtype):
    B, C, H, W = shape
    t = TYPES[dtype]
    gen = torch.Generator("cuda").manual_seed(31)
    x = torch.randn(shape, generator=gen, device="cuda")
    if place == "first":             # one value a group: at the end of the plane's first vector, or its first row
        at = 16 // t.itemsize - 1 if layout == "nchw" else 0
        x.view(B, C, -1)[:, ::C // G, at] = spike
    elif place == "anywhere":
        at = torch.randint(0, H * W, (B, G, 1), generator=gen, device="cuda")
        x.view(B, C, -1)[:, ::C // G].scatter_(2, at, spike)
    else:                            # as many as a block's first step holds, or part of them
        x.view(B, C, -1)[:, :, :11] += spike
    fmt = torch.channels_last if layout == "nhwc" else torch.contiguous_format
    x = x.to(t).contiguous(memory_format=fmt)
    gn = gb.GroupNorm(shape, G, "none", t, layout, EPS)
    y = torch.empty_like(x)
    mean, rstd = (torch.empty((B, G), device="cuda") for _ in range(2))
    gn.fwd(x, None, None, y, mean, rstd)
    wants, bounds = ref.norm_fwd(x, None, None, G, "none", EPS), ref.norm_fwd_bounds(x, None, None, G, "none", EPS)
    worst = [ref.over(got, want, bound) for got, want, bound in zip((y, mean, rstd), wants, bounds)]
    off = float(((rstd.double() - wants[2]) / wants[2]).abs().max())
    print(f"{shape} {layout} {dtype} {place} {spike:g}: y, mean, rstd {worst}, rstd off by {off:.1e}", flush=True)
    assert max(worst) <= 1, worst
