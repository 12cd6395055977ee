"""GPU: the global gradient norm and clipping against their definitions in 64 bits.

The norm is a sum in fp64, rounded once to fp32: off by 2^-24 relative, and
far less from the sum.  A clipped value is the coefficient rounded to fp32
(2^-24) times the gradient (2^-24), rounded to its type.
"""
import math

import pytest
import torch

import train_ref as ref
from backward_implicit_gemm_amd import binding as gb
from parity import Guarded

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def setup_module():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    gb.lib()


def grads(sizes, types, seed, scale=1.0, offset=0):
    gen = torch.Generator("cuda").manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        g = Guarded((n,), types[i % len(types)], offset=(offset * i) % 7)
        g.t.copy_(torch.randn(n, generator=gen, device="cuda") * scale)
        out.append(g.t)
    return out


def true_norm(gs):
    return math.sqrt(sum(float(g.double().square().sum()) for g in gs))


SIZES = [
    [1], [0], [], [5, 0, 0, 7, 0], [4096], [4095, 4097, 1], [32, 188800, 128, 147456, 3],
    [(7 * i) % 301 for i in range(97)],             # one tensor more than a launch takes
    [1 + (i * i) % 50 for i in range(250)],
    [3000001, 17, 1000003],
    [20000000],                                     # several chunks for every workgroup
]


@pytest.mark.parametrize("types", [(F32,), (BF16,), (F32, BF16, BF16)], ids=["f32", "bf16", "mixed"])
@pytest.mark.parametrize("sizes", SIZES, ids=[f"{len(s)}x{max(s, default=0)}" for s in SIZES])
def test_matches_the_definition(sizes, types):
    gs = grads(sizes, types, 1, offset=1)
    total = true_norm(gs)
    for prescale, factor in ((1.0, 0.25), (0.5, 4.0), (-2.0, 0.5)):
        guards = [Guarded(g.shape, g.dtype, offset=i % 3) for i, g in enumerate(gs)]
        clip = gb.GradClip(gs, [g.t for g in guards], prescale=prescale)
        max_norm = factor * abs(prescale) * total if total else 1.0
        norm = clip.clip(max_norm)
        torch.cuda.synchronize()
        want = abs(prescale) * total
        assert abs(float(norm) - want) <= 2 * ref.U * want
        assert float(clip.norm()) == float(norm)
        c = prescale * min(1.0, max_norm / (want + 1e-6))
        for g, o in zip(gs, guards):
            o.check("clipped gradient")
            w = g.double() * c
            assert ref.over(o.t, w, (ref.half(g.dtype) + 3 * ref.U) * w.abs() + 1e-45) <= 1


@pytest.mark.parametrize("factor", [0.25, 4.0])
def test_in_place(factor):
    gs = grads([1000, 33, 70000], (F32, BF16), 2, offset=3)
    copies = [g.clone() for g in gs]
    total = true_norm(gs)
    norm = gb.GradClip(gs).clip(factor * total)
    c = min(1.0, factor * total / (total + 1e-6))
    assert abs(float(norm) - total) <= 2 * ref.U * total
    for g, w in zip(gs, copies):
        if factor > 1:
            assert torch.equal(g, w)
        else:
            assert ref.over(g, w.double() * c, (ref.half(g.dtype) + 3 * ref.U) * w.double().abs() * c) <= 1


@pytest.mark.parametrize("scale", [1e-30, 1e30])
def test_squares_past_the_range_of_fp32(scale):
    gs = grads([5000, 3], (F32,), 3, scale=scale)
    total = true_norm(gs)
    out = [torch.empty_like(g) for g in gs]
    norm = gb.GradClip(gs, out, eps=0.0).clip(0.5 * total)
    assert abs(float(norm) - total) <= 2 * ref.U * total
    assert ref.over(out[0], gs[0].double() * 0.5, 4 * ref.U * gs[0].double().abs()) <= 1


def test_non_finite_gradients():
    for bad, finite in ((float("nan"), None), (float("inf"), 0.0)):
        gs = grads([300, 20], (F32,), 4)
        gs[1][7] = bad
        out = [torch.empty_like(g) for g in gs]
        norm = float(gb.GradClip(gs, out).clip(1.0))
        assert math.isnan(norm) if math.isnan(bad) else norm == math.inf
        assert math.isnan(float(out[1][7]))
        assert bool(torch.isnan(out[0]).all()) if finite is None else bool((out[0] == finite).all())


def test_run_to_run_graph_and_streams():
    gs = grads([100000, 33, 5000000], (F32, BF16), 5)
    out = [torch.empty_like(g) for g in gs]
    clip = gb.GradClip(gs, out)
    norm = clip.clip(1.0)
    torch.cuda.synchronize()
    want = [norm.clone()] + [o.clone() for o in out]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = clip.clip(1.0)
    side = torch.cuda.Stream()
    for rep in range(4):
        for o in out:
            o.fill_(float("nan"))
        captured.fill_(float("nan"))
        torch.cuda.synchronize()
        if rep % 2:
            with torch.cuda.stream(side):
                got = clip.clip(1.0)
        else:
            graph.replay()
            got = captured
        torch.cuda.synchronize()
        for a, b in zip([got] + out, want):
            assert torch.equal(a, b), rep


def test_present_addresses_are_used():
    """A gradient whose storage was replaced since is read where it is now."""
    g = torch.ones(1000, device="cuda")
    clip = gb.GradClip([g])
    g.data = torch.full((1000,), 2.0, device="cuda")
    norm = clip.clip(1.0)
    assert abs(float(norm) - 2 * math.sqrt(1000)) <= 1e-5
    assert float(g[0]) < 0.1
    g.data = torch.ones(999, device="cuda")
    with pytest.raises(ValueError):
        clip.clip(1.0)


def test_more_than_2_31_elements():
    g = torch.full((2 ** 31 + 5,), 0.5, dtype=BF16, device="cuda")
    g[-1] = 30000.0
    total = true_norm_chunks(g)
    norm = gb.GradClip([g]).clip(0.5 * total)
    assert abs(float(norm) - total) <= 2 * ref.U * total
    assert float(g[-1]) == pytest.approx(15000.0, rel=2 ** -8)
    assert float(g[2 ** 31]) == 0.25 and float(g[0]) == 0.25


def true_norm_chunks(g):
    return math.sqrt(sum(float(c.double().square().sum()) for c in g.split(2 ** 28)))
