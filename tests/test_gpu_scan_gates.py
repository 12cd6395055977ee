"""GPU: the gated recurrence where gates close: what is left of a large state, the value beside it and the
gradient on its way back are right in their own size, not in that of what was let go (gates_ref.py);
infinite states and values, and values near the largest fp32."""
import pytest
import torch

import train_ref
from backward_implicit_gemm_amd import binding as gb
from gates_ref import Shares

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
INF = float("inf")


def setup_module():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    gb.lib()


def run(gate, value, h0, dout, dlast, coupled=True, reset=None):
    """out, last, dgate, dvalue, dh0."""
    B, T, D = gate.shape
    h = gb.Recurrence(B, T, D, gate.dtype, coupled)
    out, dgate, dvalue = (torch.empty_like(gate) for _ in range(3))
    last, dh0 = (torch.empty((B, D), device="cuda") for _ in range(2))
    states = torch.empty(h.states_shape, device="cuda")
    h.fwd(gate, value, out, h0, last, states, reset)
    h.bwd(gate, value, states, dout, dgate, dvalue, dlast, dh0, reset)
    torch.cuda.synchronize()
    return out, last, dgate, dvalue, dh0


def plan(shape, dtype, op):
    B, T, D = shape
    s = [gb.gc_strides(T * D, D)] * 5 + [gb.gc_strides(0, 0)]
    return gb.gc_recurrence_plan_name(op, gb.gc_recurrence_desc(B, T, D, 1, *s), gb.GC_F32 if dtype == F32 else gb.GC_BF16)


# walked, walked by two channels a thread (bf16 backward), in chunks, in chunks by two channels
SHAPES = [(3, 40, 70), (2048, 20, 128), (1, 600, 70), (2, 1500, 33), (1, 800, 8000)]


def test_the_shapes_reach_what_they_are_for():
    found = {(("N=2" in plan(s, t, gb.GC_OP_BWD)), "chunks=1 " not in plan(s, t, gb.GC_OP_BWD)) for s in SHAPES for t in (F32, BF16)}
    assert found == {(False, False), (False, True), (True, False), (True, True)}


def inputs(shape, t, gates, seed):
    gen = torch.Generator("cuda").manual_seed(seed)

    def uniform(*s):
        return torch.rand(s, generator=gen, device="cuda")

    def normal(*s):
        return torch.randn(s, generator=gen, device="cuda")

    B, T, D = shape
    if gates == "any":
        gate = 50 * uniform(*shape) - 25
    elif gates == "closing":
        gate = -6 - 19 * uniform(*shape)
    else:                        # long kept, and let go now and then
        gate = torch.where(uniform(*shape) < 4 / T, -6 - 19 * uniform(*shape), 9 + normal(*shape))
    value = 10 ** (6 * uniform(*shape) - 6) * normal(*shape).sign()
    h0 = 10 ** (6 + 2 * uniform(B, D)) * normal(B, D).sign()
    # a loss at the end only
    dout = torch.zeros(shape, device="cuda")
    dout[:, -1] = normal(B, D)
    return gate.to(t), value.to(t), h0, dout.to(t), normal(B, D)


@pytest.mark.parametrize("t", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("coupled", [True, False], ids=["coupled", "not"])
@pytest.mark.parametrize("gates", ["any", "closing", "kept"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_what_is_left_is_right_in_its_own_size(shape, gates, coupled, t):
    gate, value, h0, dout, dlast = inputs(shape, t, gates, sum(shape))
    got = run(gate, value, h0, dout, dlast, coupled)
    ref = Shares(gate, value, h0, coupled)
    want = [ref.stored(t), (ref.last, ref.d_last), *ref.backward(dout, dlast, t)]
    for name, g, w in zip(("out", "last", "dgate", "dvalue", "dh0"), got, want):
        e = train_ref.over(g, *w)
        assert e <= 1.0, (name, e)


@pytest.mark.parametrize("T", [3, 900], ids=["walked", "chunks"])
def test_single_gates(T):
    """A large state meets one closing gate at the last step."""
    f = torch.tensor([-10.0, -16.0, -17.0, -20.0, -40.0, -100.0, -INF, -16.0, -20.0], device="cuda")
    h0 = torch.tensor([1e3, 100.0, 1e8, 1e3, 1e8, 1e8, 1e6, 100.0, -1e3], device="cuda")[None]
    v = torch.tensor([0.3, 1e-6, 0.7, 1e-6, 0.7, 0.7, 1e-3, 0.0, 1e-6], device="cuda")
    D = f.numel()
    gate = torch.full((1, T, D), 80.0, device="cuda")      # keeps all: 1 - a is 1.8e-35
    value = torch.zeros((1, T, D), device="cuda")
    gate[0, -1], value[0, -1] = f, v
    dlast = torch.linspace(0.7, 1.7, D, device="cuda")[None]
    for coupled in (True, False):
        got = run(gate, value, h0, torch.zeros_like(gate), dlast, coupled)
        a, i = torch.sigmoid(f.double()), torch.sigmoid(-f.double())
        last = a * h0[0].double() + (i if coupled else 1.0) * v.double()
        dh0 = a * dlast[0].double()
        # the exponential 1.5|f| + 3, and 12 more roundings; what underflows is 0
        rel = (1.5 * f.double().abs().clamp(max=88) + 15) * train_ref.U
        floor = 2.0 ** -126 * (h0[0].double().abs() + 2)
        assert bool(((got[1][0].double() - last).abs() <= rel * (a * h0[0].double().abs() + v.double().abs()) + floor).all())
        assert bool(((got[4][0].double() - dh0).abs() <= rel * dh0 + floor).all())


def same_kind(got, want):
    """Infinities with their sign and NaN at the same places."""
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.isinf(got), torch.isinf(want))
    inf = torch.isinf(want)
    assert torch.equal(got.double()[inf], want.double()[inf])


def steps(gate, value, h0, dout, dlast, reset, coupled):
    """The definition one step at a time, in 64 bits."""
    f, v, d = gate.double(), value.double(), dout.double()
    a, i = torch.sigmoid(f), torch.sigmoid(-f)
    T = f.shape[1]
    h, out, before = h0.double(), torch.empty_like(f), torch.empty_like(f)
    for t in range(T):
        before[:, t] = h if reset is None else h.masked_fill(reset[:, t, None], 0.0)
        h = out[:, t] = a[:, t] * before[:, t] + (i[:, t] if coupled else 1.0) * v[:, t]
    back, dv = dlast.double(), torch.empty_like(f)
    for t in range(T - 1, -1, -1):
        g = back + d[:, t]
        dv[:, t] = i[:, t] * g if coupled else g
        back = a[:, t] * g if reset is None else (a[:, t] * g).masked_fill(reset[:, t, None], 0.0)
    return out, h, dv, back


@pytest.mark.parametrize("t", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("coupled", [True, False], ids=["coupled", "not"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_infinities_stay(shape, coupled, t):
    """An infinite state, value or gradient goes on as it does in the definition, also against its opposite (NaN)."""
    B, T, D = shape
    gen = torch.Generator("cuda").manual_seed(9)
    gate = (12 * torch.rand(shape, generator=gen, device="cuda") - 6).to(t)
    value = torch.randn(shape, generator=gen, device="cuda").to(t)
    dout = torch.randn(shape, generator=gen, device="cuda").to(t)
    h0, dlast = (torch.randn((B, D), generator=gen, device="cuda") for _ in range(2))
    b, m = B - 1, T // 2
    h0[b, 0], h0[b, 3] = INF, -INF
    value[b, m, 5], value[b, m, 6], value[b, T - 1, 3] = INF, -INF, INF
    value[b, m, 9] = float("nan")
    dlast[b, 10], dout[b, m, 11], dout[b, m, 12] = INF, -INF, float("nan")
    dout[b, 1, 10] = -INF
    reset = torch.rand((B, T), generator=gen, device="cuda") < 0.2 / T
    reset[b] = reset[:, 0] = False
    if B > 1:
        reset[0, T // 3], h0[0, 2], dlast[0, 4] = True, INF, INF
    for r in (None, reset):
        got = run(gate, value, h0, dout, dlast, coupled, r)
        out, last, dv, dh0 = steps(gate, value, h0, dout, dlast, r, coupled)
        for g, w in ((got[0], out), (got[1], last), (got[3], dv), (got[4], dh0)):
            same_kind(g, w)
        # finite where the state and the gradient are
        assert torch.equal(torch.isfinite(got[2]).all(1), (torch.isfinite(out) & torch.isfinite(dv)).all(1) & torch.isfinite(h0))


@pytest.mark.parametrize("T", [20, 700], ids=["walked", "chunks"])
def test_values_near_the_largest(T):
    """States and values of opposite sign whose difference is past fp32's largest."""
    gen = torch.Generator("cuda").manual_seed(10)
    shape = (1, T, 40)
    gate = 6 * torch.rand(shape, generator=gen, device="cuda") - 3
    value = 3e38 * torch.randn(shape, generator=gen, device="cuda").sign()
    h0 = 3e38 * torch.randn((1, 40), generator=gen, device="cuda").sign()
    dout, dlast = torch.zeros(shape, device="cuda"), torch.ones((1, 40), device="cuda")
    dout[:, ::5] = 0.25
    got = run(gate, value, h0, dout, dlast)
    ref = Shares(gate, value, h0, True)
    want = [ref.stored(F32), (ref.last, ref.d_last), *ref.backward(dout, dlast, F32)]
    for name, g, w in zip(("out", "last", "dgate", "dvalue", "dh0"), got, want):
        e = train_ref.over(g, *w)
        assert e <= 1.0, (name, e)
