"""GPU: distillation from a teacher's top logits against its definition in 64 bits, with
bounds derived per element (core_ref.py)."""
import pytest
import torch

import core_ref as ref
from backward_implicit_gemm_amd import binding as gb
from parity import Guarded
from test_gpu_rows import Part

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
INF = float("inf")


def setup_module():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    gb.lib()


def problem(rows, V, K, t, seed=0, index=torch.int32, teacher=F32, extra=0, offset=0, masked=0.0, empty=0.0, twice=False):
    gen = torch.Generator("cuda").manual_seed(seed)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    z = 2 * torch.randn((rows, V), generator=gen, device="cuda")
    if masked:
        bar = uniform(rows, V) < masked
        bar[:, 0] = False
        z = z.masked_fill(bar, -INF)
    # random places, several of them the same where `twice`, else each once while there are enough
    places = (uniform(rows, K) * V).long().clamp_(max=V - 1) if twice or K > V else uniform(rows, V).topk(K, 1).indices
    tl = 3 * torch.randn((rows, K), generator=gen, device="cuda")
    if masked:
        tl = tl.masked_fill(z.gather(1, places) == -INF, -INF)
    if empty:
        places[uniform(rows) < empty] = -1
        places[uniform(rows, K) < empty] = V
    dloss = uniform(rows) - 0.3
    return Part(rows, V, t, extra, offset, z), Wide(places.to(index), extra), Part(rows, K, teacher, extra, offset, tl), dloss


class Wide:
    """Whole numbers as rows that are parts of wider ones."""

    def __init__(self, values, extra):
        self.t = torch.zeros((values.shape[0], values.shape[1] + extra), dtype=values.dtype, device="cuda")[:, :values.shape[1]]
        self.t.copy_(values)


def close(got, value, bound, name):
    both = torch.isfinite(value)
    assert torch.equal(torch.isfinite(got), both), name
    e = ref.over(torch.where(both, got.double(), 0.0), torch.where(both, value, 0.0), torch.where(both, bound, 1.0))
    assert e <= 1.0, (name, e)


def check(rows, V, K, t, tau=1.0, in_place=False, **kw):
    z, index, teacher, dloss = problem(rows, V, K, t, **kw)
    extra, offset = kw.get("extra", 0), kw.get("offset", 0)
    (loss, d_loss), (peak, mass, d_mass), (dz, d_dz) = ref.distill(z.t, index.t, teacher.t, tau, dloss, t)
    h = gb.Distill(rows, V, K, t, tau, teacher.t.dtype)
    got = [Guarded((rows,), F32) for _ in range(4)]
    h.fwd(z.t, index.t, teacher.t, *(g.t for g in got[:3]))
    grads = [Part(rows, V, t, extra and extra + 1, offset) for _ in range(2)]
    keep = z.t.clone()
    if in_place:
        grads[0] = z
    h.bwd(z.t, index.t, teacher.t, got[1].t, got[2].t, dloss, grads[0].t)
    torch.cuda.synchronize()
    if in_place:
        grads[0] = Part(rows, V, t, 0, 0, z.t)
        z.t.copy_(keep)
        grads[1] = z
    h.step(z.t, index.t, teacher.t, dloss, got[3].t, grads[1].t)
    torch.cuda.synchronize()
    for g in got + grads:
        g.check("outputs")
    close(got[0].t, loss, d_loss, "loss")
    close(got[3].t, loss, d_loss, "loss of the step")
    assert torch.equal(got[1].t.double(), peak)
    close(got[2].t, mass, d_mass, "mass")
    close(grads[0].t, dz, d_dz, "dlogits")
    close(grads[1].t, dz, d_dz, "dlogits of the step")


# one logit, rows of lanes, ends inside a vector, workgroups, every number of held vectors, rows that are walked
SHAPES = [(1, 1, 1), (5, 2, 1), (3, 3, 7), (70, 7, 3), (1000, 18, 4), (33, 63, 10), (9, 65, 64), (300, 300, 8), (17, 515, 100),
          (64, 1025, 20), (6, 2049, 256), (5, 4100, 33), (3, 9000, 64), (2, 20001, 1024), (3, 33000, 64), (2, 40961, 64),
          (2, 50257, 5), (1, 80000, 70), (2, 99999, 64), (1, 140000, 300)]


@pytest.mark.parametrize("t", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_against_the_definition(shape, t):
    check(*shape, t)
    check(*shape, t, seed=1, tau=2.0, masked=0.2, empty=0.2, index=torch.int64)


@pytest.mark.parametrize("t", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", [(40, 5, 9), (30, 300, 50), (9, 3001, 33), (3, 30011, 700)], ids=str)
def test_entries_of_one_place(shape, t):
    check(*shape, t, twice=True, empty=0.1)


@pytest.mark.parametrize("t", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", [(40, 5, 2), (30, 301, 8), (9, 3001, 33), (3, 30011, 70), (2, 131077, 9)], ids=str)
def test_parts_of_wider_rows_and_in_place(shape, t):
    check(*shape, t, extra=5, offset=3, teacher=BF16)
    check(*shape, t, in_place=True, tau=0.7, twice=True)


@pytest.mark.parametrize("V", [50, 5000, 150000])
def test_rows_without_entries(V):
    """No loss and no gradient, whatever the row's logits hold."""
    rows, K = 6, 4
    z = torch.randn((rows, V), device="cuda")
    z[0], z[1, 3], z[2, 0] = -INF, float("nan"), INF
    index = torch.arange(K, dtype=torch.int32, device="cuda").repeat(rows, 1)
    teacher = torch.zeros((rows, K), device="cuda")
    index[0], index[1] = -1, V
    teacher[2] = -INF
    index[3, :2], teacher[3, 2:] = -2 ** 31, -INF
    h = gb.Distill(rows, V, K, F32)
    loss, peak, mass, again = (torch.full((rows,), 9.0, device="cuda") for _ in range(4))
    grads = [torch.full((rows, V), 9.0, device="cuda") for _ in range(2)]
    dloss = torch.ones(rows, device="cuda")
    dloss[1] = float("nan")
    h.fwd(z, index, teacher, loss, peak, mass)
    h.bwd(z, index, teacher, peak, mass, dloss, grads[0])
    h.step(z, index, teacher, dloss, again, grads[1])
    torch.cuda.synchronize()
    for t in (loss[:4], again[:4], grads[0][:4], grads[1][:4]):
        assert bool((t == 0).all())
    for t in (loss[4:], again[4:], grads[0][4:], grads[1][4:]):
        assert bool((t != 0).any(-1).all()) and bool(torch.isfinite(t).all())


@pytest.mark.parametrize("V", [50, 5000, 150000])
def test_masks(V):
    """Logits of the type's lowest value count as any other; a masked place that the teacher has a share
    of has an infinite loss and a gradient; NaN stays in its row."""
    rows, K = 5, 3
    low = torch.finfo(F32).min
    z = torch.full((rows, V), low, device="cuda")
    z[1, 7], z[2] = 0.0, 0.0
    z[2, 1], z[3, 40] = -INF, float("nan")
    index = torch.tensor([[7, 8, 9]] * rows, dtype=torch.int32, device="cuda")
    index[2] = torch.tensor([1, 2, 2])
    index[1] = torch.tensor([7, -1, -1])
    teacher = torch.zeros((rows, K), device="cuda")
    h = gb.Distill(rows, V, K, F32)
    loss, peak, mass, again = (torch.empty(rows, device="cuda") for _ in range(4))
    grads = [torch.empty((rows, V), device="cuda") for _ in range(2)]
    dloss = torch.ones(rows, device="cuda")
    h.fwd(z, index, teacher, loss, peak, mass)
    h.bwd(z, index, teacher, peak, mass, dloss, grads[0])
    h.step(z, index, teacher, dloss, again, grads[1])
    torch.cuda.synchronize()
    for ls, g in ((loss, grads[0]), (again, grads[1])):
        # all alike: a uniform softmax; log(V / 3) of it, to the rounding of log and of the sums
        want = float(torch.log(torch.tensor(V / 3, dtype=torch.float64)))
        assert abs(float(ls[0]) - want) <= 60 * ref.U * want
        assert abs(float(g[0, 0]) * V - 1) <= 60 * ref.U
        assert float(ls[1]) == 0.0 and float(g[1].abs().max()) == 0.0
        assert float(ls[2]) == INF and abs(float(g[2, 1]) + 1 / 3) <= 8 * ref.U
        assert abs(float(g[2, 2]) - (1 / (V - 1) - 2 / 3)) <= 60 * ref.U and bool(torch.isfinite(g[2]).all())
        assert bool(torch.isnan(ls[3])) and bool(torch.isnan(g[3]).all())
        assert bool(torch.isfinite(g[4]).all())


def test_gradient_against_differences():
    rows, V, K, tau = 2, 13, 5, 1.7
    z, index, teacher, dloss = problem(rows, V, K, F32, twice=True)
    h = gb.Distill(rows, V, K, F32, tau)
    loss, dz = torch.empty(rows, device="cuda"), torch.empty((rows, V), device="cuda")
    h.step(z.t, index.t, teacher.t, dloss, loss, dz)
    torch.cuda.synchronize()
    for e in range(rows * V):
        v = []
        for d in (1e-4, -1e-4):
            x = z.t.double().clone()
            x.view(-1)[e] += d
            v.append(float((ref.distill(x, index.t, teacher.t, tau, dloss, F32)[0][0] * dloss.double()).sum()))
        diff = (v[0] - v[1]) / 2e-4
        assert abs(diff - float(dz.view(-1)[e])) <= 2e-6, e


def test_no_rows():
    e = torch.empty((0, 9), device="cuda")
    i, t, r = torch.empty((0, 2), dtype=torch.int64, device="cuda"), torch.empty((0, 2), device="cuda"), torch.empty(0, device="cuda")
    h = gb.Distill(0, 9, 2, F32)
    h.fwd(e, i, t, r, r, r)
    h.bwd(e, i, t, r, r, r, e)
    h.step(e, i, t, r, r, e)


@pytest.mark.parametrize("shape", [(100, 300, 8), (20, 40961, 64), (2, 150001, 64)], ids=str)
def test_bit_reproducible(shape):
    z, index, teacher, dloss = problem(*shape, BF16, twice=True)
    h = gb.Distill(*shape, BF16)

    def once():
        r = [torch.empty(shape[0], device="cuda") for _ in range(4)]
        g = [torch.empty(shape[:2], dtype=BF16, device="cuda") for _ in range(2)]
        h.fwd(z.t, index.t, teacher.t, *r[:3])
        h.bwd(z.t, index.t, teacher.t, r[1], r[2], dloss, g[0])
        h.step(z.t, index.t, teacher.t, dloss, r[3], g[1])
        return r + g

    first = once()
    for _ in range(3):
        for a, b in zip(first, once()):
            assert torch.equal(a, b)
