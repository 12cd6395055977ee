"""GPU: the gated recurrence's kernels in the combinations that the planner's shapes alone do not run: sequences of
their own lengths walked by two channels a thread, every instance with and without resets in both forms,
and resets, lengths and both forms where a wave's sequences lie 4 GiB apart."""
import pytest
import torch

import core_ref as ref
from backward_implicit_gemm_amd import binding as gb
from test_gpu_core_instances import FAR, TYPES, of, parts
from test_gpu_scan import check, close, problem

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def setup_module():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    gb.lib()


def plan(B, T, D, t, op):
    s = [gb.gc_strides(T * D, D)] * 5 + [gb.gc_strides(T, 1)]
    return gb.gc_recurrence_plan_name(op, gb.gc_recurrence_desc(B, T, D, 1, *s), gb.GC_F32 if t == F32 else gb.GC_BF16)


def spread_lengths(B, T):
    """All of it, nothing, one step, one off a block, and what lies between."""
    return [(T, 0, 1, T - 1, T // 2, 17, 16, 15, T // 3, T)[i % 10] for i in range(B)]


# walked: several sequences a wave, whole waves, a wave and one lane (with an odd and an even number of channels)
WALKED = [(6600, 20, 40), (6700, 37, 39), (2048, 20, 128), (2049, 21, 129), (2050, 18, 130)]
# in chunks, ends inside and before chunks; odd and even
CHUNKS = [(3, 400, 8001), (3, 401, 8000), (1, 1300, 4999)]


@pytest.mark.parametrize("shape", WALKED + CHUNKS, ids=str)
def test_two_channels_a_thread_with_lengths(shape):
    B, T, D = shape
    name = plan(B, T, D, BF16, gb.GC_OP_BWD)
    assert "N=2" in name and ("chunks=1 " in name) == (shape in WALKED), name
    lengths = spread_lengths(B, T) if B > 3 else [T, T * 3 // 8, 0][:B] if B > 1 else [T - 150]
    check(B, T, D, BF16, lengths=lengths)
    check(B, T, D, BF16, coupled=False, lengths=lengths, reset=0.02, layout="tb", seed=2)


@pytest.mark.parametrize("case", of("scan"), ids=str)
def test_both_forms_with_and_without_resets(case):
    """What the instances' own test leaves: coupled without resets, not coupled with them, and lengths."""
    op, dtype, B, T, D = case
    check(B, T, D, TYPES[dtype], coupled=True)
    check(B, T, D, TYPES[dtype], coupled=False, reset=0.01, layout="tb", seed=3)
    check(B, T, D, TYPES[dtype], coupled=True, lengths=spread_lengths(B, T), ends=False, seed=4)


@pytest.mark.parametrize("t", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("coupled", [True, False], ids=["coupled", "not"])
@pytest.mark.parametrize("T", [21, 300], ids=["walked", "chunks"])
def test_far_apart_with_resets_and_lengths(T, coupled, t):
    B, D = 3, 10
    p = problem(B, T, D, t, reset=0.05, lengths=[T, T // 2 + 1, 1])
    far = parts((B, T, D), (FAR + 64, D, 1), t, 6)
    gate, value, out, dout, dgate, dvalue = far
    for a, k in ((gate, "gate"), (value, "value"), (dout, "dout")):
        a.copy_(p[k].t)
    h = gb.Recurrence(B, T, D, t, coupled)
    for reset in (None, p["reset"]):
        states, last, dh0 = torch.empty(h.states_shape, device="cuda"), *(torch.empty((B, D), device="cuda") for _ in range(2))
        h.fwd(gate, value, out, p["h0"], last, states, reset, p["lengths"])
        h.bwd(gate, value, states, dout, dgate, dvalue, p["dlast"], dh0, reset, p["lengths"])
        torch.cuda.synchronize()
        scan = ref.Scan(p["gate"].t, p["value"].t, p["h0"], reset, p["lengths"], coupled)
        close(out, scan.stored(t), "out")
        close(last, (scan.last, scan.d_last), "last")
        for got, want, name in zip((dgate, dvalue, dh0), scan.backward(p["dout"].t, p["dlast"], t), ("dgate", "dvalue", "dh0")):
            close(got, want, name)


def test_the_most_chunks():
    """256 chunks, whose carry holds 16 a wave, with states that reach through all of them."""
    B, T, D = 1, 2 * 16 * 256, 5
    for op, t in ((gb.GC_OP_FWD, F32), (gb.GC_OP_BWD, BF16)):
        assert "chunks=256 " in plan(B, T, D, t, op)
    check(B, T, D, F32, keep=14.0)
    check(B, T - 5, D, BF16, keep=14.0, coupled=False, seed=1)
