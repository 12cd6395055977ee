"""GPU: what a helper allocates by itself follows the stream of the call.

A call is enqueued behind a wait on a side stream and its result and helper are
dropped at once: no memory of theirs may come back to the current stream before the
call has run.  The buffers taken there afterwards keep their contents, and the call's
outputs are right.  A captured call does not need its helper any more.
"""
import pytest
import torch

from backward_implicit_gemm_amd import binding as gb

pytestmark = pytest.mark.gpu


def setup_module():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    gb.lib()


def clip():
    g = [torch.full((3000,), 2.0, device="cuda"), torch.ones(41, device="cuda")]
    out = [torch.zeros_like(t) for t in g]
    return (lambda: gb.GradClip(g, out)), (lambda h, s: h.clip(0.5, stream=s) is None), out


def norm():
    g = [torch.full((3000,), 2.0, device="cuda")]
    return (lambda: gb.GradClip(g)), (lambda h, s: h.norm(stream=s) is None), []


def embedding():
    tok = torch.arange(9000, device="cuda", dtype=torch.int32).reshape(90, 100) * 7 % 5000
    dout = torch.arange(9000 * 24, device="cuda").remainder(13).float().reshape(90, 100, 24)
    out = torch.zeros((5000, 24), device="cuda")
    return (lambda: gb.Embedding(90, 100, 5000, 24, torch.float32)), (lambda h, s: h.bwd(tok, dout, out, stream=s)), [out]


def small_table():
    tok = torch.arange(9000, device="cuda", dtype=torch.int64).reshape(90, 100) * 7 % 50
    dout = torch.arange(9000 * 24, device="cuda").remainder(13).float().reshape(90, 100, 24)
    out = torch.zeros((50, 24), device="cuda")
    return (lambda: gb.Embedding(90, 100, 50, 24, torch.float32)), (lambda h, s: h.bwd(tok, dout, out, stream=s)), [out]


def group_norm(shape, G):
    def make():
        x = torch.arange(shape[0] * shape[1] * shape[2] * shape[3], device="cuda").remainder(37).float().reshape(shape)
        dy = x.remainder(5)
        y, dx = torch.zeros_like(x), torch.zeros_like(x)
        p = [torch.zeros(shape[1], device="cuda") for _ in range(2)]
        st = [torch.zeros((shape[0], G), device="cuda") for _ in range(2)]

        def call(h, s):
            h.fwd(x, None, None, y, *st, stream=s)
            h.bwd(x, None, None, dy, *st, dx, *p, stream=s)

        return (lambda: gb.GroupNorm(shape, G, "silu", torch.float32)), call, [y, dx, *p, *st]
    return make


CALLS = {"clip": clip, "norm": norm, "embedding": embedding, "small table": small_table,
         "resident norm": group_norm((300, 32, 3, 4), 4), "split norm": group_norm((2, 16, 200, 200), 2)}


def fresh():
    """Buffers of many sizes on the current stream, and the byte they are filled with."""
    return [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for k in range(4, 24) for n in [1 << k] * 3]


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


def test_results_of_side_streams():
    """The norm belongs to the call's stream: it is right after that stream, whatever the current one allocates."""
    g = [torch.full((400,), 3.0, device="cuda")]
    h, side = gb.GradClip(g), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(5_000_000)
    norm = h.norm(stream=side)
    buffers = fresh()
    side.synchronize()
    assert float(norm) == 60.0
    torch.cuda.synchronize()
    assert all(bool((b == 0x5A).all()) for b in buffers)
    default = h.norm(stream=torch.cuda.default_stream())
    with torch.cuda.stream(side):
        again = h.norm(stream=torch.cuda.default_stream().cuda_stream)
    torch.cuda.synchronize()
    assert float(default) == 60.0 and float(again) == 60.0


@pytest.mark.parametrize("call", sorted(CALLS))
def test_a_captured_call_outlives_its_helper(call):
    make, run, outs = CALLS[call]()
    run(make(), None)
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    h = make()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(h, None)
    del h
    buffers = fresh()
    for rep in range(3):
        for o in outs:
            o.fill_(-1.0)
        run(make(), None)       # eager work between the replays
        torch.cuda.synchronize()
        for o in outs:
            o.fill_(-1.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(bool((b == 0x5A).all()) for b in buffers), rep
        for o, w in zip(outs, want):
            assert torch.equal(o, w), rep
