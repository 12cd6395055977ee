"""GPU: layer norm of a residual stream against its definition in 64 bits, with bounds
derived per element (core_ref.py)."""
import pytest
import torch

import core_ref as ref
from backward_implicit_gemm_amd import binding as gb
from parity import Guarded

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TYPES = [(F32, F32), (BF16, F32), (BF16, BF16)]
IDS = ["f32", "bf16", "bf16 params"]


def setup_module():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    gb.lib()


def normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


class Part:
    """Rows that are parts of wider ones, `extra` values of a sentinel between them."""

    def __init__(self, rows, dim, dtype, extra=0, offset=0, values=None):
        self.g = Guarded((rows * (dim + extra),), dtype, offset=offset)
        self.wide = self.g.t.view(rows, dim + extra)
        self.t = self.wide[:, :dim]
        self.between = self.wide[:, dim:].clone()
        if values is not None:
            self.t.copy_(values)

    def check(self, name):
        self.g.check(name)
        bits = torch.int32 if self.t.dtype == F32 else torch.int16
        assert torch.equal(self.wide[:, self.t.shape[1]:].contiguous().view(bits), self.between.contiguous().view(bits)), name


def inputs(rows, dim, t, pt, seed, extra=0, offset=0, shift=0.5):
    gen = torch.Generator("cuda").manual_seed(seed)
    x = Part(rows, dim, t, extra, offset, normal(gen, rows, dim) * (0.3 + torch.rand(dim, generator=gen, device="cuda")) + shift)
    res = Part(rows, dim, t, extra and extra + 2, offset, 2 * normal(gen, rows, dim))
    dy = Part(rows, dim, t, extra and extra + 1, offset, normal(gen, rows, dim))
    gamma, beta = (1 + 0.2 * normal(gen, dim)).to(pt), (0.2 * normal(gen, dim)).to(pt)
    return x, res, dy, gamma, beta


def close(got, want, name):
    value, bound = want
    e = ref.over(got, value, bound)
    assert e <= 1.0, (name, e)


def check_fwd(rows, dim, t, pt, seed=0, residual=True, extra=0, offset=0, shift=0.5, eps=1e-5, params=True, in_place=False):
    x, res, _, gamma, beta = inputs(rows, dim, t, pt, seed, extra, offset, shift)
    if not params:
        gamma = beta = None
    r = res.t.clone() if residual else None
    want = ref.rows_fwd(x.t, r, gamma, beta, eps, t)
    y = Part(rows, dim, t, extra and extra + 3, offset)
    total = res if in_place else Part(rows, dim, t, extra and extra + 4, offset)
    mean, rstd = Guarded((rows,), F32), Guarded((rows,), F32)
    h = gb.LayerNorm(rows, dim, t, eps, pt)
    h.fwd(x.t, gamma, beta, y.t, mean.t, rstd.t, res.t if residual else None, total.t if residual else None)
    torch.cuda.synchronize()
    for g, w, name in ((y, want[0], "y"), (mean, want[1], "mean"), (rstd, want[2], "rstd")):
        g.check(name)
        close(g.t, w, name)
    if residual:
        total.check("total")
        close(total.t, want[3], "total")
    return h, y.t


def check_bwd(rows, dim, t, pt, seed=0, dtotal=True, extra=0, offset=0, params=True, sums=(True, True), in_place=None):
    x, res, dy, gamma, _ = inputs(rows, dim, t, pt, seed, extra, offset)
    if not params:
        gamma = None
    v = x.t.double()
    mean = v.mean(1).float()
    rstd = (v.var(1, correction=0) + 1e-5).rsqrt().float()
    want = ref.rows_bwd(x.t, gamma, dy.t.clone(), mean, rstd, res.t.clone() if dtotal else None, t, pt)
    dx = {None: lambda: Part(rows, dim, t, extra and extra + 3, offset), "dtotal": lambda: res, "dy": lambda: dy}[in_place]()
    dgamma, dbeta = (Guarded((dim,), pt) if s else None for s in sums)
    h = gb.LayerNorm(rows, dim, t, 1e-5, pt)
    h.bwd(x.t, gamma, dy.t, mean, rstd, dx.t, *(None if g is None else g.t for g in (dgamma, dbeta)),
          res.t if dtotal else None)
    torch.cuda.synchronize()
    for g, w, name in ((dx, want[0], "dx"), (dgamma, want[1], "dgamma"), (dbeta, want[2], "dbeta")):
        if g is not None:
            g.check(name)
            close(g.t, w, name)


# short rows, every vector count of a thread, ends inside a vector, several waves, walked rows
SHAPES = [(1, 1), (3, 2), (700, 3), (65, 7), (1, 8), (33, 9), (5, 63), (2, 64), (129, 100), (1, 1760), (300, 1760), (7, 2047),
          (64, 2049), (40, 4096), (3, 5001), (9, 8200), (2, 12000), (2, 16384), (3, 16385), (2, 70001), (5000, 40), (2500, 300)]


@pytest.mark.parametrize("types", TYPES, ids=IDS)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(shape, types):
    check_fwd(*shape, *types, residual=True)
    check_fwd(*shape, *types, seed=1, residual=False, params=False)


@pytest.mark.parametrize("types", TYPES, ids=IDS)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward(shape, types):
    check_bwd(*shape, *types, dtotal=True)
    check_bwd(*shape, *types, seed=1, dtotal=False, params=False)


@pytest.mark.parametrize("types", TYPES, ids=IDS)
@pytest.mark.parametrize("shape", [(37, 5), (50, 131), (20, 1760), (6, 9001), (3, 20001)], ids=str)
def test_parts_of_wider_rows(shape, types):
    check_fwd(*shape, *types, extra=5, offset=3)
    check_bwd(*shape, *types, extra=5, offset=3)


@pytest.mark.parametrize("t", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", [(37, 5), (50, 131), (20, 1761), (6, 9001), (3, 20001)], ids=str)
def test_in_place(shape, t):
    check_fwd(*shape, t, F32, in_place=True)
    check_bwd(*shape, t, F32, in_place="dtotal")
    check_bwd(*shape, t, F32, in_place="dy", extra=3)


@pytest.mark.parametrize("sums", [(True, False), (False, True), (False, False)], ids=str)
def test_optional_sums(sums):
    check_bwd(70, 130, F32, F32, sums=sums)
    check_bwd(5, 17000, F32, F32, sums=sums)


def test_a_mean_far_from_zero():
    """The squares are taken around the mean: an offset of 2000 widths costs no more than its own rounding."""
    check_fwd(30, 1760, F32, F32, shift=2000.0)
    check_fwd(3, 20000, F32, F32, shift=2000.0)


def test_no_rows():
    h = gb.LayerNorm(0, 12, F32)
    e, s = torch.empty((0, 12), device="cuda"), torch.empty(0, device="cuda")
    h.fwd(e, None, None, e, s, s)
    dgamma, dbeta = (torch.full((12,), 7.0, device="cuda") for _ in range(2))
    h.bwd(e, None, e, s, s, e, dgamma, dbeta)
    torch.cuda.synchronize()
    assert bool((dgamma == 0).all()) and bool((dbeta == 0).all())


def test_rows_with_non_finite_values_leave_the_others():
    x = torch.ones((6, 100), device="cuda")
    x[:, ::2] = -1.0
    y, clean = torch.empty_like(x), torch.empty_like(x)
    h = gb.LayerNorm(6, 100, F32)
    h.fwd(x, None, None, clean)
    x[1, 3], x[4, 99] = float("nan"), float("inf")
    h.fwd(x, None, None, y)
    torch.cuda.synchronize()
    assert bool(torch.isnan(y[1]).all()) and bool(torch.isnan(y[4]).all())
    for r in (0, 2, 3, 5):
        assert torch.equal(y[r], clean[r])


@pytest.mark.parametrize("shape", [(1000, 1760), (31, 130), (4, 20000)], ids=str)
def test_bit_reproducible(shape):
    x, res, dy, gamma, beta = inputs(*shape, BF16, F32, 3)
    h = gb.LayerNorm(*shape, BF16)
    mean, rstd = (torch.empty(shape[0], device="cuda") for _ in range(2))

    def once():
        y, total, dx = (torch.empty(shape, dtype=BF16, device="cuda") for _ in range(3))
        dg, db = (torch.empty(shape[1], device="cuda") for _ in range(2))
        h.fwd(x.t, gamma, beta, y, mean, rstd, res.t, total)
        h.bwd(total, gamma, dy.t, mean, rstd, dx, dg, db, res.t)
        return y, total, dx, dg, db

    first = once()
    for _ in range(3):
        for a, b in zip(first, once()):
            assert torch.equal(a, b)


def test_gradient_against_differences():
    """dx, dgamma and dbeta against central differences of the 64-bit forward, whose own error is the
    step's square (1e-8) and rounding over step (1e-12)."""
    gen = torch.Generator("cuda").manual_seed(5)
    rows, D = 3, 11
    x, dy, gamma, beta = (normal(gen, *s) for s in ((rows, D), (rows, D), (D,), (D,)))
    h = gb.LayerNorm(rows, D, F32)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = (torch.empty(rows, device="cuda") for _ in range(2))
    dgamma, dbeta = torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
    h.fwd(x, gamma, beta, y, mean, rstd)
    h.bwd(x, gamma, dy, mean, rstd, dx, dgamma, dbeta)
    torch.cuda.synchronize()

    def loss(x, gamma, beta):
        return float((ref.rows_fwd(x, None, gamma, beta, 1e-5, torch.float64)[0][0] * dy.double()).sum())

    args = [x.double(), gamma.double(), beta.double()]
    for k, got in enumerate((dx, dgamma, dbeta)):
        for e in range(0, got.numel(), 2):
            step = [a.clone() for a in args], [a.clone() for a in args]
            step[0][k].view(-1)[e] += 1e-4
            step[1][k].view(-1)[e] -= 1e-4
            diff = (loss(*step[0]) - loss(*step[1])) / 2e-4
            # fp32 results of sums of up to 33 values of a few units
            assert abs(diff - float(got.view(-1)[e])) <= 2e-5 * (1 + abs(diff)), (k, e)
