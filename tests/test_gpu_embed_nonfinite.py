"""GPU: a non-finite gradient in the small-table form leaves the slabs of 32 columns
that do not hold it with the bits they have without it.

The last slab of a row that is no multiple of 32 long shares columns with the one
before; both are summed, one in another order where it meets a non-finite value, and only
one of them may be written.
"""
import pytest
import torch

from backward_implicit_gemm_amd import binding as gb

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def setup_module():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    gb.lib()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("V,D", [(300, 33), (100, 40), (60, 95), (128, 64), (30, 31), (30, 2)])
def test_other_slabs_keep_their_bits(V, D, dtype, bad):
    t = TYPES[dtype]
    rows, T = 300, 20
    gen = torch.Generator("cuda").manual_seed(21)
    tok = torch.randint(0, V, (rows, T), generator=gen, device="cuda", dtype=torch.int32)
    dout = torch.randn((rows, T, D), generator=gen, device="cuda").to(t)
    e = gb.Embedding(rows, T, V, D, t)
    assert gb.gc_embed_plan_name(e.desc, e.dt) == "embed_grad_onehot"

    def gradient(d):
        out = torch.full((V, D), -7.0, dtype=t, device="cuda")
        e.bwd(tok, d, out)
        return out

    bits = torch.int32 if t == torch.float32 else torch.int16
    clean = gradient(dout)
    for c in sorted({0, D - 1, (D - 1) // 32 * 32, min(31, D - 1)}):
        spoilt = dout.clone()
        spoilt[5, 3, c] = bad
        got = gradient(spoilt)
        # columns written by a workgroup that holds column c: its slab's, and the last slab's,
        # which begins 32 columns before the end
        at = torch.arange(D, device="cuda")
        meets = at // 32 == c // 32
        if c >= D - 32:
            meets |= at >= (D - 1) // 32 * 32
        assert torch.equal(got[:, ~meets].view(bits), clean[:, ~meets].view(bits)), c
        assert not bool(torch.isfinite(got[tok[5, 3], c]))
        assert int((~torch.isfinite(got)).sum()) == 1
        for _ in range(3):
            assert torch.equal(gradient(spoilt).view(bits), got.view(bits)), c
