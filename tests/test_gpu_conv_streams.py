"""GPU: a convolution's workspace follows the stream of the call.

A call on a side stream that still waits, its helper dropped at once: the workspace must
not come back to the current stream before the call has run.
"""
import pytest
import torch

from backward_implicit_gemm_amd import binding as gb
from test_gpu_streams import fresh

pytestmark = pytest.mark.gpu


def setup_module():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    gb.lib()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("how", ["argument", "current", "captured"])
def test_dropped_while_a_side_stream_still_runs(how, dtype):
    xs, ws, stride = (64, 59, 11, 15), (128, 59, 5, 5), 3
    gen = torch.Generator("cuda").manual_seed(3)
    x, w = (torch.randn(s, generator=gen, device="cuda").to(dtype) for s in (xs, ws))
    shape = gb.Conv(xs, ws, stride, 0, dtype).y_shape
    dy = torch.randn(shape, generator=gen, device="cuda").to(dtype)
    outs = [torch.zeros(s, dtype=dtype, device="cuda") for s in (shape, xs, ws)]

    def run(c, stream):
        c.fwd(x, w, outs[0], stream=stream)
        c.bwd(x, w, dy, None, outs[1], outs[2], stream=stream)

    run(gb.Conv(xs, ws, stride, 0, dtype), None)
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    c = gb.Conv(xs, ws, stride, 0, dtype)
    for o in outs:
        o.fill_(-1.0)
    torch.cuda.synchronize()
    if how == "captured":
        with torch.cuda.graph(graph):
            run(c, None)
    else:
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
            if how == "current":
                run(c, None)
        if how == "argument":
            run(c, side)
    del c
    buffers = fresh()
    for rep in range(3 if how == "captured" else 1):
        if how == "captured":
            run(gb.Conv(xs, ws, stride, 0, dtype), None)
            torch.cuda.synchronize()
            for o in outs:
                o.fill_(-1.0)
            graph.replay()
        torch.cuda.synchronize()
        assert all(bool((b == 0x5A).all()) for b in buffers), "memory of the call was given away while it was in use"
        for o, v in zip(outs, want):
            assert torch.equal(o, v), rep
