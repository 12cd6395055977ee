"""GPU: each kernel instance that the recurrent core's planners pick, against the definition; and
tensors whose parts lie 4 GiB and more apart."""
import pytest
import torch

import core_instances
import core_ref as ref
from backward_implicit_gemm_amd import binding as gb
from test_gpu_distill import check as check_distill
from test_gpu_rows import check_bwd, check_fwd
from test_gpu_scan import check as check_scan

pytestmark = pytest.mark.gpu

FOUND = core_instances.instances()
TYPES = {gb.GC_F32: torch.float32, gb.GC_BF16: torch.bfloat16}


def setup_module():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    gb.lib()


def of(kind):
    return sorted((v for k, v in FOUND.items() if k[0] == kind), key=str)


@pytest.mark.parametrize("case", of("rows"), ids=str)
def test_rows(case):
    op, dtype, rows, D = case
    for more in (False, True):
        if op == gb.GC_OP_FWD:
            check_fwd(rows, D, TYPES[dtype], torch.float32, residual=more)
        else:
            check_bwd(rows, D, TYPES[dtype], torch.float32, dtotal=more)


@pytest.mark.parametrize("case", of("scan"), ids=str)
def test_scan(case):
    op, dtype, B, T, D = case
    check_scan(B, T, D, TYPES[dtype], coupled=True, reset=0.01)
    check_scan(B, T, D, TYPES[dtype], coupled=False, layout="tb")


@pytest.mark.parametrize("case", of("distill"), ids=str)
def test_distill(case):
    op, dtype, rows, V, K = case
    for k in (min(K, 16), max(K, 17)):      # written again, and looked up
        check_distill(rows, V, k, TYPES[dtype], twice=True, empty=0.05)


# ------------------------------------------------------ offsets past 32 bits --
FAR = 1 << 31          # elements: 4 GiB of bf16, 8 GiB of fp32


def parts(shape, strides, dtype, count):
    """`count` tensors of far strides side by side in one buffer."""
    reach = sum((n - 1) * s for n, s in zip(shape, strides)) + 1
    room = 1 << 16
    buf = torch.empty(reach + count * room, dtype=dtype, device="cuda")
    return [buf[i * room:].as_strided(shape, strides) for i in range(count)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("far", ["batch", "step"])
def test_recurrence_far_apart(far, dtype):
    B, T, D = (3, 19, 10) if far == "batch" else (5, 3, 10)
    strides = (FAR + 64, D, 1) if far == "batch" else (D, FAR + 64, 1)
    f, v, out, d, dg, dv = parts((B, T, D), strides, dtype, 6)
    gen = torch.Generator("cuda").manual_seed(3)
    near = [torch.randn((B, T, D), generator=gen, device="cuda").to(dtype) for _ in range(3)]
    for a, b in zip((f, v, d), near):
        a.copy_(b)
    h, got = gb.Recurrence(B, T, D, dtype), []
    for x in ((f, v, out, d, dg, dv), (*near[:2], *(torch.empty_like(near[0]) for _ in range(1)), near[2],
                                       *(torch.empty_like(near[0]) for _ in range(2)))):
        states, last = torch.empty(h.states_shape, device="cuda"), torch.empty((B, D), device="cuda")
        h.fwd(x[0], x[1], x[2], None, last, states)
        h.bwd(x[0], x[1], states, x[3], x[4], x[5])
        torch.cuda.synchronize()
        got.append([t.clone() for t in (x[2], x[4], x[5], last)])
    for a, b in zip(*got):
        assert torch.equal(a, b)
    scan = ref.Scan(*near[:2], None, None, None, True)
    value, bound = scan.stored(dtype)
    assert ref.over(got[0][0], value, bound) <= 1.0


def test_layer_norm_far_apart():
    rows, D = 3, 100
    x, res, y, total, dy, dx = parts((rows, D), (FAR + 64, 1), torch.bfloat16, 6)
    gen = torch.Generator("cuda").manual_seed(4)
    near = [torch.randn((rows, D), generator=gen, device="cuda").bfloat16() for _ in range(3)]
    for a, b in zip((x, res, dy), near):
        a.copy_(b)
    h, stats = gb.LayerNorm(rows, D, torch.bfloat16), [torch.empty(rows, device="cuda") for _ in range(2)]
    h.fwd(x, None, None, y, *stats, res, total)
    h.bwd(total, None, dy, *stats, dx, dtotal=res)
    torch.cuda.synchronize()
    want = ref.rows_fwd(near[0], near[1], None, None, 1e-5, torch.bfloat16)
    for got, w in zip((y, *stats, total), want):
        assert ref.over(got, *w) <= 1.0
    want = ref.rows_bwd(total.contiguous(), None, near[2], *stats, near[1], torch.bfloat16, torch.float32)
    assert ref.over(dx, *want[0]) <= 1.0


def test_distillation_far_apart():
    rows, V, K = 3, 700, 20
    z, dz = parts((rows, V), (FAR + 64, 1), torch.bfloat16, 2)
    gen = torch.Generator("cuda").manual_seed(5)
    near = (2 * torch.randn((rows, V), generator=gen, device="cuda")).bfloat16()
    z.copy_(near)
    teacher, index = (2 * torch.randn((rows, V), generator=gen, device="cuda")).topk(K, 1)
    loss, dloss = torch.empty(rows, device="cuda"), torch.ones(rows, device="cuda")
    gb.Distill(rows, V, K, torch.bfloat16).step(z, index, teacher, dloss, loss, dz)
    torch.cuda.synchronize()
    (value, bound), _, (grad, d_grad) = ref.distill(near, index, teacher, 1.0, dloss, torch.bfloat16)
    assert ref.over(loss, value, bound) <= 1.0 and ref.over(dz, grad, d_grad) <= 1.0


def test_masked_rows_with_a_teacher():
    """A row of nothing but -inf: every q is 0, the loss infinite, the gradient minus the teacher's shares."""
    for V, K in ((60, 2), (60, 20), (5000, 2), (5000, 20), (170000, 20)):
        z = torch.full((2, V), -float("inf"), device="cuda")
        index = torch.arange(K, device="cuda").repeat(2, 1)
        teacher = torch.zeros((2, K), device="cuda")
        h = gb.Distill(2, V, K, torch.float32)
        loss, peak, mass, again = (torch.empty(2, device="cuda") for _ in range(4))
        dloss = torch.ones(2, device="cuda")
        g = [torch.empty_like(z) for _ in range(2)]
        h.fwd(z, index, teacher, loss, peak, mass)
        h.bwd(z, index, teacher, peak, mass, dloss, g[0])
        h.step(z, index, teacher, dloss, again, g[1])
        torch.cuda.synchronize()
        assert bool((loss == float("inf")).all()) and bool((again == float("inf")).all())
        assert bool((mass == 0).all())
        for t in g:
            # one division by K, one product
            assert bool(((t[:, :K] + 1 / K).abs() <= 4 * ref.U / K).all()) and bool((t[:, K:] == 0).all())
