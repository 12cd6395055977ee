"""GPU: what the recurrent core's helpers allocate by themselves follows the stream of the call, as
the other helpers' does; captured calls outlive their helper, and two of them share nothing."""
import pytest
import torch

from backward_implicit_gemm_amd import binding as gb
from test_gpu_streams import fresh

pytestmark = pytest.mark.gpu


def setup_module():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    gb.lib()


def values(*shape, mod=37):
    n = 1
    for s in shape:
        n *= s
    return torch.arange(n, device="cuda").remainder(mod).float().reshape(shape) / mod - 0.4


def layer_norm(rows, D):
    def make():
        x, dy = values(rows, D), values(rows, D, mod=11)
        y, dx, total = (torch.zeros_like(x) for _ in range(3))
        p = [torch.zeros(D, device="cuda") for _ in range(2)]
        st = [torch.zeros(rows, device="cuda") for _ in range(2)]

        def call(h, s):
            h.fwd(x, None, None, y, *st, dy, total, stream=s)
            h.bwd(total, None, dy, *st, dx, *p, x, stream=s)

        return (lambda: gb.LayerNorm(rows, D, torch.float32)), call, [y, dx, total, *p, *st]
    return make


def recurrence(B, T, D):
    def make():
        f, v, d = values(B, T, D) * 5, values(B, T, D, mod=13), values(B, T, D, mod=11)
        out, dg, dv = (torch.zeros_like(f) for _ in range(3))
        h = gb.Recurrence(B, T, D, torch.float32)
        states, last, dh0, h0 = torch.zeros(h.states_shape, device="cuda"), *(torch.zeros((B, D), device="cuda") for _ in range(3))

        def call(h, s):
            h.fwd(f, v, out, h0, last, states, stream=s)
            h.bwd(f, v, states, d, dg, dv, None, dh0, stream=s)

        return (lambda: gb.Recurrence(B, T, D, torch.float32)), call, [out, last, states, dg, dv, dh0]
    return make


def distill(rows, V, K):
    def make():
        z, dloss = values(rows, V) * 9, values(rows) + 1
        index = (torch.arange(rows * K, device="cuda") * 7919 % V).reshape(rows, K)
        teacher = values(rows, K, mod=5)
        loss, peak, mass, again = (torch.zeros(rows, device="cuda") for _ in range(4))
        g = [torch.zeros_like(z) for _ in range(2)]

        def call(h, s):
            h.fwd(z, index, teacher, loss, peak, mass, stream=s)
            h.bwd(z, index, teacher, peak, mass, dloss, g[0], stream=s)
            h.step(z, index, teacher, dloss, again, g[1], stream=s)

        return (lambda: gb.Distill(rows, V, K, torch.float32)), call, [loss, peak, mass, again, *g]
    return make


CALLS = {"rows": layer_norm(300, 130), "long rows": layer_norm(3, 17000), "walk": recurrence(200, 20, 70),
         "chunks": recurrence(1, 3000, 33), "distill": distill(50, 300, 8), "long distill": distill(3, 90001, 70)}


@pytest.mark.parametrize("how", ["argument", "raw handle", "current"])
@pytest.mark.parametrize("call", sorted(CALLS))
def test_dropped_while_a_side_stream_still_runs(call, how):
    make, run, outs = CALLS[call]()
    run(make(), None)
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    for o in outs:
        o.fill_(-1.0)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    h = make()
    if how == "current":
        with torch.cuda.stream(side):
            run(h, None)
    else:
        run(h, side if how == "argument" else side.cuda_stream)
    del h
    buffers = fresh()
    torch.cuda.synchronize()
    assert all(bool((b == 0x5A).all()) for b in buffers), "memory of the call was given away while it was in use"
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


@pytest.mark.parametrize("call", sorted(CALLS))
def test_captured_calls_outlive_their_helper_and_share_nothing(call):
    """Two graphs of one helper, replayed on two streams at once, and eager calls between the replays."""
    make, run, outs = CALLS[call]()
    second, run2, outs2 = CALLS[call]()
    run(make(), None)
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    h = make()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for graph, body in zip(graphs, (run, run2)):
        with torch.cuda.graph(graph):
            for _ in range(3):
                body(h, None)
    del h
    buffers = fresh()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for rep in range(3):
        run(make(), None)
        torch.cuda.synchronize()
        for o in outs + outs2:
            o.fill_(-1.0)
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        assert all(bool((b == 0x5A).all()) for b in buffers), rep
        for got in (outs, outs2):
            for o, w in zip(got, want):
                assert torch.equal(o, w), rep


@pytest.mark.parametrize("call", sorted(CALLS))
def test_helpers_leave_no_cycle(call):
    """A dropped helper's memory is free at once, without a collection."""
    import gc
    import weakref
    make = CALLS[call]()[0]
    gc.collect()
    gc.disable()
    try:
        h = make()
        ref = weakref.ref(h)
        del h
        assert ref() is None
    finally:
        gc.enable()
