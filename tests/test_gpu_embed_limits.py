"""GPU: the longest rows and the tallest table an embedding takes.

dim and vocab go up to 2^31 - 1, where (dim + 7) / 8 and vocab + 255 no longer fit an
int.  One token copies (or adds up) one row, so a product with a power of two is exact.
"""
import pytest
import torch

from backward_implicit_gemm_amd import binding as gb

pytestmark = pytest.mark.gpu

MOST = 2 ** 31 - 1


def setup_module():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    gb.lib()


@pytest.mark.parametrize("dim", [MOST, MOST - 3])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_longest_rows(dtype, dim):
    row = torch.arange(1, 252, device="cuda").repeat(dim // 251 + 1)[:dim].to(dtype)
    e = gb.Embedding(1, 1, 1, dim, dtype, 0.5)
    tok = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    out = torch.full((1, 1, dim), -1.0, dtype=dtype, device="cuda")
    e.fwd(tok, row[None], out)
    row.mul_(0.5)
    assert torch.equal(out[0, 0], row)
    dtable = torch.full((1, dim), -1.0, dtype=dtype, device="cuda")
    e.bwd(tok, out, dtable)
    row.mul_(0.5)
    assert torch.equal(dtable[0], row)
    tok.fill_(1)
    e.bwd(tok, out, dtable)
    assert not bool(dtable.any())


def test_tallest_table():
    V, T = MOST, 5000
    gen = torch.Generator("cuda").manual_seed(2)
    tok = torch.randint(0, V, (1, T), generator=gen, device="cuda", dtype=torch.int64).sort().values
    tok[0, 0], tok[0, -1], tok[0, -2] = 0, V - 1, V
    e = gb.Embedding(1, T, V, 1, torch.bfloat16)
    dout = torch.arange(T, device="cuda").remainder(7).add(1).bfloat16().reshape(1, T, 1)
    dtable = torch.full((V, 1), -1.0, dtype=torch.bfloat16, device="cuda")
    e.bwd(tok, dout, dtable)
    at, place = tok[tok < V].unique(return_inverse=True)
    want = torch.zeros(at.numel(), device="cuda").index_add_(0, place, dout[tok < V][:, 0].float()).bfloat16()
    assert torch.equal(dtable[at, 0], want)
    assert int(dtable.count_nonzero()) == at.numel()
    out = torch.empty_like(dout)
    e.fwd(tok, dtable, out)
    assert torch.equal(out[0, tok[0] < V, 0], want[place]) and not bool(out[0, tok[0] >= V].any())
