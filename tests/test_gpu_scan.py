"""GPU: the gated recurrence against its definition in 64 bits, step by step, with bounds
derived per element (core_ref.py)."""
import pytest
import torch

import core_ref as ref
from backward_implicit_gemm_amd import binding as gb
from parity import Guarded

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def setup_module():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    gb.lib()


class Seqs:
    """Sequences in one of several layouts of one guarded buffer: (batch, length, dim) views."""

    def __init__(self, B, T, D, dtype, layout="bt", offset=0):
        if layout in ("bt", "tb"):
            self.g = Guarded((B * T * D,), dtype, offset=offset)
            self.t = self.g.t.view(B, T, D) if layout == "bt" else self.g.t.view(T, B, D).transpose(0, 1)
        else:                    # a part of wider rows, time first
            self.g = Guarded((B * T * (2 * D + 3),), dtype, offset=offset)
            self.t = self.g.t.view(T, B, 2 * D + 3)[..., D + 1:2 * D + 1].transpose(0, 1)

    def fill(self, values):
        self.t.copy_(values)
        return self


def problem(B, T, D, t, seed=0, layout="bt", offset=0, reset=0.0, lengths=None, keep=3.0):
    gen = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    p = {"gate": Seqs(B, T, D, t, layout, offset).fill(normal(B, T, D) * 1.5 + keep * torch.rand(D, generator=gen, device="cuda")),
         "value": Seqs(B, T, D, t, layout, offset).fill(normal(B, T, D)),
         "dout": Seqs(B, T, D, t, layout, offset).fill(normal(B, T, D)),
         "h0": normal(B, D), "dlast": normal(B, D), "reset": None, "lengths": None}
    if reset:
        p["reset"] = torch.rand((B, T), generator=gen, device="cuda") < reset
        if layout != "bt":
            p["reset"] = p["reset"].t().contiguous().t()
    if lengths is not None:
        p["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    return p


def close(got, want, name):
    value, bound = want
    e = ref.over(got, value, torch.where(bound == 0, 1e-300, bound))
    assert e <= 1.0, (name, e)


def check(B, T, D, t, coupled=True, layout="bt", offset=0, ends=True, **kw):
    p = problem(B, T, D, t, layout=layout, offset=offset, **kw)
    h0, dlast = (p["h0"], p["dlast"]) if ends else (None, None)
    h = gb.Recurrence(B, T, D, t, coupled)
    out = Seqs(B, T, D, t, layout, offset)
    last, states = Guarded((B, D), F32), Guarded(h.states_shape, F32)
    h.fwd(p["gate"].t, p["value"].t, out.t, h0, last.t, states.t, p["reset"], p["lengths"])
    dgate, dvalue = Seqs(B, T, D, t, layout, offset), Seqs(B, T, D, t, layout, offset)
    dh0 = Guarded((B, D), F32)
    h.bwd(p["gate"].t, p["value"].t, states.t, p["dout"].t, dgate.t, dvalue.t, dlast, dh0.t, p["reset"], p["lengths"])
    torch.cuda.synchronize()
    scan = ref.Scan(p["gate"].t, p["value"].t, h0, p["reset"], p["lengths"], coupled)
    close(out.t, scan.stored(t), "out")
    close(last.t, (scan.last, scan.d_last), "last")
    want = scan.backward(p["dout"].t, dlast, t)
    for got, w, name in ((dgate.t, want[0], "dgate"), (dvalue.t, want[1], "dvalue"), (dh0.t, want[2], "dh0")):
        close(got, w, name)
    for g in (out.g, last, states, dgate.g, dvalue.g, dh0):
        g.check("outputs")
    if layout == "part":         # what lies between the parts is as it was
        for s in (out, dgate, dvalue):
            wide = s.g.t.view(T, B, -1)
            bits = torch.int32 if t == F32 else torch.int16
            other = torch.cat([wide[..., :D + 1], wide[..., 2 * D + 1:]], -1).contiguous().view(bits)
            assert bool((other == s.g.pat).all())


# steps around a block of 16, one channel, odd channels; several chunks; many sequences
SHAPES = [(1, 1, 1), (3, 1, 8), (64, 1, 512), (2, 2, 3), (1, 15, 5), (2, 16, 2), (2, 17, 64), (5, 33, 130), (1, 100, 1),
          (1, 1000, 4), (2, 777, 33), (1, 2049, 129), (3, 300, 777), (700, 20, 65), (33, 64, 512)]


@pytest.mark.parametrize("t", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_against_the_definition(shape, t):
    check(*shape, t)
    check(*shape, t, coupled=False, ends=False, seed=1)


@pytest.mark.parametrize("t", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("layout", ["tb", "part"])
@pytest.mark.parametrize("shape", [(4, 1, 6), (5, 40, 33), (2, 700, 129), (1, 1500, 1)], ids=str)
def test_layouts(shape, layout, t):
    check(*shape, t, layout=layout, offset=1, reset=0.05)


@pytest.mark.parametrize("t", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("coupled", [True, False], ids=["coupled", "not"])
def test_resets_and_lengths(coupled, t):
    lengths = [50, 0, 1, 15, 16, 17, 49, 32]
    check(8, 50, 37, t, coupled, lengths=lengths)
    check(8, 50, 37, t, coupled, reset=0.2, lengths=lengths, layout="tb")
    check(8, 50, 36, t, coupled, reset=1.0)
    # chunks that end within, before and behind the sequences, with resets in some of them
    check(3, 3000, 20, t, coupled, reset=0.002, lengths=[3000, 1111, 0])
    check(3, 3000, 21, t, coupled, reset=0.3, lengths=[2999, 64, 2048])


@pytest.mark.parametrize("t", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("D", [63, 64, 65, 129, 130, 200])
def test_lengths_around_a_wave(D, t):
    """Channels that leave a wave partly empty or nearly so, sequences that end in different chunks."""
    check(4, 700, D, t, lengths=[700, 333, 0, 16], reset=0.01)
    check(4, 90, D, t, lengths=[90, 33, 64, 1], layout="tb")


def test_lengths_outside_the_steps_are_taken_into_them():
    B, T, D = 4, 20, 6
    p = problem(B, T, D, F32)
    h = gb.Recurrence(B, T, D, F32)
    outs = []
    for lengths in ([-5, 100, 2 ** 31 - 1, 20], [0, 20, 20, 20]):
        out, last = torch.empty((B, T, D), device="cuda"), torch.empty((B, D), device="cuda")
        h.fwd(p["gate"].t, p["value"].t, out, p["h0"], last, None, None, torch.tensor(lengths, dtype=torch.int32, device="cuda"))
        outs.append((out, last))
    torch.cuda.synchronize()
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    assert torch.equal(outs[0][1][0], p["h0"][0])


@pytest.mark.parametrize("t", [F32, BF16], ids=["f32", "bf16"])
def test_a_packed_row_is_its_sequences(t):
    """Sequences one behind the other in a row, with a reset at each start, are the sequences alone."""
    lengths, D = [40, 1, 100, 16, 143], 24
    T = sum(lengths)
    p = problem(1, T, D, t)
    reset = torch.zeros((1, T), dtype=torch.uint8, device="cuda")
    starts = [sum(lengths[:i]) for i in range(len(lengths))]
    reset[0, starts] = 1
    h = gb.Recurrence(1, T, D, t)
    out = torch.empty((1, T, D), dtype=t, device="cuda")
    h.fwd(p["gate"].t, p["value"].t, out, torch.full((1, D), float("nan"), device="cuda"), None, None, reset)
    for s, n in zip(starts, lengths):
        alone = torch.empty((1, n, D), dtype=t, device="cuda")
        gb.Recurrence(1, n, D, t).fwd(p["gate"].t[:, s:s + n], p["value"].t[:, s:s + n], alone)
        scan = ref.Scan(p["gate"].t[:, s:s + n], p["value"].t[:, s:s + n], None, None, None, True)
        torch.cuda.synchronize()
        close(out[:, s:s + n], scan.stored(t), "packed")
        close(alone, scan.stored(t), "alone")


@pytest.mark.parametrize("T", [60, 4000], ids=["walked", "chunks"])
def test_not_finite_until_a_reset(T):
    """What is not finite stays in its channel, until a reset, forward and backward."""
    B, D, at, cut = 2, 40, T // 3, T // 2 + 1
    p = problem(B, T, D, F32)
    reset = torch.zeros((B, T), dtype=torch.bool, device="cuda")
    reset[0, cut] = True
    h = gb.Recurrence(B, T, D, F32)
    p["value"].t[0, at, 3] = float("inf")
    p["value"].t[0, at, 5] = float("nan")
    p["dout"].t[0, at + 2, 9] = float("nan")
    out, states = torch.empty((B, T, D), device="cuda"), torch.empty(h.states_shape, device="cuda")
    dgate, dvalue = torch.empty_like(out), torch.empty_like(out)
    last, dh0 = (torch.empty((B, D), device="cuda") for _ in range(2))
    h.fwd(p["gate"].t, p["value"].t, out, p["h0"], last, states, reset)
    h.bwd(p["gate"].t, p["value"].t, states, p["dout"].t, dgate, dvalue, p["dlast"], dh0, reset)
    torch.cuda.synchronize()
    bad = ~torch.isfinite(out)
    want = torch.zeros_like(bad)
    want[0, at:cut, 3] = want[0, at:cut, 5] = True
    assert torch.equal(bad, want)
    assert bool(torch.isfinite(last).all())
    want = torch.zeros_like(bad)
    want[0, :at + 3, 9] = True
    assert torch.equal(~torch.isfinite(dvalue), want)
    assert bool(torch.isnan(dh0[0, 9])) and int((~torch.isfinite(dh0)).sum()) == 1


def test_gates_at_their_ends():
    """Gates of +-inf and far beyond exp's range keep all or take all; NaN stays."""
    gate = torch.tensor([float("-inf"), -1e30, -200.0, -100.0, 100.0, 1e30, float("inf"), float("nan")], device="cuda")
    B, T, D = 1, 3, 8
    value = torch.arange(1.0, 4.0, device="cuda").reshape(1, 3, 1).expand(B, T, D).contiguous()
    h0 = torch.full((B, D), 7.0, device="cuda")
    h = gb.Recurrence(B, T, D, F32)
    out, states = torch.empty((B, T, D), device="cuda"), torch.empty(h.states_shape, device="cuda")
    f = gate.expand(B, T, D)          # distances of 0
    dgate, dvalue, dh0 = torch.empty_like(out), torch.empty_like(out), torch.empty_like(h0)
    h.fwd(f, value, out, h0, None, states)
    h.bwd(f, value, states, torch.ones_like(out), dgate, dvalue, None, dh0)
    torch.cuda.synchronize()
    for c in range(4):
        assert out[0, :, c].tolist() == [1.0, 2.0, 3.0] and dvalue[0, :, c].tolist() == [1.0] * 3
    for c in range(4, 7):
        assert out[0, :, c].tolist() == [7.0] * 3 and bool((dvalue[0, :, c].abs() < 1e-40).all())
        assert float(dh0[0, c]) == 3.0
    assert bool((dgate[..., :7].abs() < 1e-30).all())
    assert bool(torch.isnan(out[..., 7]).all()) and bool(torch.isnan(dgate[..., 7]).all())


@pytest.mark.parametrize("t", [F32, BF16], ids=["f32", "bf16"])
def test_steps_one_at_a_time(t):
    """A policy that acts: one step a call, the state in place, is the whole sequence."""
    B, T, D = 9, 21, 50
    p = problem(B, T, D, t, layout="tb", reset=0.1)
    state, one = p["h0"].clone(), gb.Recurrence(B, 1, D, t)
    out = torch.empty((B, T, D), dtype=t, device="cuda")
    for s in range(T):
        one.fwd(p["gate"].t[:, s:s + 1], p["value"].t[:, s:s + 1], out[:, s:s + 1], state, state, None, p["reset"][:, s:s + 1])
    torch.cuda.synchronize()
    scan = ref.Scan(p["gate"].t, p["value"].t, p["h0"], p["reset"], None, True)
    close(out, scan.stored(t), "out")
    close(state, (scan.last, scan.d_last), "state")


def test_ends_in_place_and_left_out():
    """last over h0, dh0 over dlast, walked and in chunks; without them the rest is the same."""
    for B, T, D in ((40, 30, 65), (1, 3000, 33)):
        p = problem(B, T, D, F32)
        h = gb.Recurrence(B, T, D, F32)

        def once(h0, last, dlast, dh0, keep=True):
            out, dg, dv = (torch.empty((B, T, D), device="cuda") for _ in range(3))
            states = torch.empty(h.states_shape, device="cuda")
            h.fwd(p["gate"].t, p["value"].t, out, h0, last, states)
            if not keep:
                again = torch.empty_like(out)
                h.fwd(p["gate"].t, p["value"].t, again, h0)
                assert torch.equal(out, again)
            h.bwd(p["gate"].t, p["value"].t, states, p["dout"].t, dg, dv, dlast, dh0)
            torch.cuda.synchronize()
            return out, dg, dv

        last, dh0 = torch.empty((B, D), device="cuda"), torch.empty((B, D), device="cuda")
        want = once(p["h0"], last, p["dlast"], dh0)
        for a, b in zip(want, once(p["h0"], None, p["dlast"], None, keep=False)):
            assert torch.equal(a, b)
        x, y = p["h0"].clone(), p["dlast"].clone()
        for a, b in zip(want, once(x, x, y, y)):
            assert torch.equal(a, b)
        assert torch.equal(x, last) and torch.equal(y, dh0)


def test_no_steps_and_no_sequences():
    h0, dlast = torch.randn((3, 7), device="cuda"), torch.randn((3, 7), device="cuda")
    e, last, dh0 = torch.empty((3, 0, 7), device="cuda"), torch.zeros((3, 7), device="cuda"), torch.zeros((3, 7), device="cuda")
    h = gb.Recurrence(3, 0, 7, F32)
    h.fwd(e, e, e, h0, last, torch.empty(h.states_shape, device="cuda"))
    h.bwd(e, e, torch.empty(h.states_shape, device="cuda"), e, e, e, dlast, dh0)
    torch.cuda.synchronize()
    assert torch.equal(last, h0) and torch.equal(dh0, dlast)
    e = torch.empty((0, 5, 7), device="cuda")
    none = torch.empty((0, 7), device="cuda")
    gb.Recurrence(0, 5, 7, F32).fwd(e, e, e, none, none)


def test_a_long_memory_is_not_worn_off():
    """A state that keeps 1 - 4e-6 of itself a step, over 20,000 steps: 64-bit result to fp32's bound."""
    B, T, D = 1, 20000, 3
    gate = torch.full((B, T, D), 12.5, device="cuda")
    value = torch.zeros((B, T, D), device="cuda")
    h0, out, last = torch.ones((B, D), device="cuda"), torch.empty((B, T, D), device="cuda"), torch.empty((B, D), device="cuda")
    gb.Recurrence(B, T, D, F32).fwd(gate, value, out, h0, last)
    torch.cuda.synchronize()
    want = float(torch.sigmoid(torch.tensor(12.5, dtype=torch.float64)) ** T)
    # 1 - a is off by (3 * 12.5 + 12) U relative, which the 20,000 steps multiply by 20000 * 3.7e-6 = 0.075;
    # each step rounds the state once (U), in chunks twice
    assert abs(float(last[0, 0]) / want - 1) <= 0.075 * 50 * ref.U + 2 * T * ref.U


def test_gradient_against_differences():
    """Central differences of the 64-bit recurrence (error of the step's square, 1e-8)."""
    B, T, D = 2, 19, 3
    p = problem(B, T, D, F32, reset=0.1, lengths=[19, 11])
    h = gb.Recurrence(B, T, D, F32)
    out, dgate, dvalue = (torch.empty((B, T, D), device="cuda") for _ in range(3))
    states, dh0 = torch.empty(h.states_shape, device="cuda"), torch.empty((B, D), device="cuda")
    h.fwd(p["gate"].t, p["value"].t, out, p["h0"], None, states, p["reset"], p["lengths"])
    h.bwd(p["gate"].t, p["value"].t, states, p["dout"].t, dgate, dvalue, p["dlast"], dh0, p["reset"], p["lengths"])
    torch.cuda.synchronize()

    def loss(gate, value, h0):
        s = ref.Scan(gate, value, h0, p["reset"], p["lengths"], True)
        return float((s.out * p["dout"].t.double()).sum() + (s.last * p["dlast"].double()).sum())

    args = [p["gate"].t.double(), p["value"].t.double(), p["h0"].double()]
    for k, got in enumerate((dgate, dvalue, dh0)):
        for e in range(0, got.numel(), 7):
            step = [a.clone() for a in args], [a.clone() for a in args]
            step[0][k].view(-1)[e] += 1e-4
            step[1][k].view(-1)[e] -= 1e-4
            diff = (loss(*step[0]) - loss(*step[1])) / 2e-4
            assert abs(diff - float(got.reshape(-1)[e])) <= 2e-5 * (1 + abs(diff)), (k, e)


@pytest.mark.parametrize("shape", [(20, 100, 65), (1, 5000, 129)], ids=str)
def test_bit_reproducible(shape):
    p = problem(*shape, BF16, reset=0.01)
    h = gb.Recurrence(*shape, BF16)

    def once():
        out, dg, dv = (torch.empty(shape, dtype=BF16, device="cuda") for _ in range(3))
        states = torch.empty(h.states_shape, device="cuda")
        h.fwd(p["gate"].t, p["value"].t, out, p["h0"], None, states, p["reset"])
        h.bwd(p["gate"].t, p["value"].t, states, p["dout"].t, dg, dv, p["dlast"], None, p["reset"])
        return out, dg, dv, states

    first = once()
    for _ in range(3):
        for a, b in zip(first, once()):
            assert torch.equal(a, b)
