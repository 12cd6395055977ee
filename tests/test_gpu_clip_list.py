"""GPU: clipping refuses a gradient whose type, device or layout has changed
since the helper was made, before anything reads it.
"""
import pytest
import torch

from backward_implicit_gemm_amd import binding as gb

pytestmark = pytest.mark.gpu


def setup_module():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    gb.lib()


@pytest.mark.parametrize("change", [
    lambda t: t.bfloat16(), lambda t: t.view(torch.int32), lambda t: t.cpu(), lambda t: torch.ones(2000, device="cuda")[::2],
], ids=["type", "type of the same width", "device", "strided"])
@pytest.mark.parametrize("which", ["gradient", "output"])
def test_refuses_changed_tensors(which, change):
    grads = [torch.ones(1000, device="cuda"), torch.ones(7, device="cuda")]
    out = [torch.zeros_like(g) for g in grads]
    clip = gb.GradClip(grads, out)
    t = (grads if which == "gradient" else out)[0]
    t.data = change(t.data)
    with pytest.raises(ValueError, match="has changed"):
        clip.clip(1.0)
    with pytest.raises(ValueError, match="has changed"):
        clip.norm()


def test_module_that_changes_its_type():
    m = torch.nn.Linear(64, 33, device="cuda")
    m(torch.ones((2, 64), device="cuda")).sum().backward()
    clip = gb.GradClip([p.grad for p in m.parameters()])
    clip.clip(1.0)
    m.bfloat16()
    with pytest.raises(ValueError, match="has changed"):
        clip.clip(1.0)
    norm = gb.GradClip([p.grad for p in m.parameters()]).clip(1.0)
    assert abs(float(norm) - 1) < 1e-2


def test_replaced_memory_and_flags_are_taken():
    g = torch.ones(1000, device="cuda")
    clip = gb.GradClip([g])
    g.requires_grad_()
    g.data = torch.full((10, 100), 2.0, device="cuda")
    for _ in range(2):
        assert abs(float(clip.norm()) - 2 * 1000 ** 0.5) <= 1e-5
