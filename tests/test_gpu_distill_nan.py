"""GPU: distillation of rows that hold NaN or +inf beside masked logits: the softmax of such a row is NaN at every
place, so its loss is NaN and so is its gradient everywhere, whichever threads hold the masked ones."""
import pytest
import torch

from backward_implicit_gemm_amd import binding as gb

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
INF, NAN = float("inf"), float("nan")


def setup_module():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    gb.lib()


@pytest.mark.parametrize("t", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("K", [3, 20])
@pytest.mark.parametrize("V", [5, 40, 300, 5000, 40961, 200003])
def test_not_a_number_beside_masked_logits(V, K, t):
    # the odd one out at either end, over rows of nothing else, of one more logit, of all the others
    rows, bad = [], []
    for odd in (NAN, INF):
        for at in (0, V - 1):
            for fill in ("masked", "one", "all"):
                z = torch.linspace(-3, 3, V, device="cuda") if fill == "all" else torch.full((V,), -INF, device="cuda")
                if fill == "one":
                    z[V // 2] = 1.0
                z[at] = odd
                rows.append(z)
                bad.append(True)
    ordinary = torch.full((V,), -INF, device="cuda")
    ordinary[V // 3] = 2.0
    rows.append(ordinary)
    bad.append(False)
    z = torch.stack(rows).to(t)
    n = z.shape[0]
    # entries at masked places too; in the last row at the only logit
    index = (torch.arange(K, device="cuda") * 2 % V).repeat(n, 1)
    index[-1] = V // 3
    teacher = torch.linspace(0, 1, K, device="cuda").repeat(n, 1)
    h = gb.Distill(n, V, K, t)
    loss, peak, mass, again = (torch.empty(n, device="cuda") for _ in range(4))
    dloss, grads = torch.ones(n, device="cuda"), [torch.empty_like(z) for _ in range(2)]
    h.fwd(z, index, teacher, loss, peak, mass)
    h.bwd(z, index, teacher, peak, mass, dloss, grads[0])
    h.step(z, index, teacher, dloss, again, grads[1])
    torch.cuda.synchronize()
    want = torch.tensor(bad, device="cuda")
    for got in (loss, again):
        assert torch.equal(torch.isnan(got), want)
    for got in grads:
        assert torch.equal(torch.isnan(got).all(1), want)
        # one logit that takes it all, and a teacher who says the same
        assert bool((got[-1].abs() <= 2.0 ** -20).all())
