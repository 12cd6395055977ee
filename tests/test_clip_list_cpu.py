"""The list of tensors a clipping call reads by address: its memory may be
replaced between calls, nothing else about it.  Runs without a GPU.
"""
import pytest
import torch

from backward_implicit_gemm_amd import binding as gb


def tensors():
    return [torch.zeros(6), torch.zeros((3, 4), dtype=torch.bfloat16), torch.zeros(0), torch.zeros(())]


def test_addresses_are_the_present_ones():
    ts = tensors()
    held = gb._Tensors(ts)
    assert held.addresses() == [t.data_ptr() for t in ts]
    new = torch.ones(6)
    ts[0].data = new
    assert held.addresses()[0] == new.data_ptr()
    assert gb._Tensors([]).addresses() == []


def test_what_leaves_the_memory_the_same_is_taken():
    ts = tensors()
    held = gb._Tensors(ts)
    ts[0].requires_grad_()
    ts[1].data = torch.zeros((2, 6), dtype=torch.bfloat16)
    with torch.inference_mode():
        assert held.addresses() == [t.data_ptr() for t in ts]
    assert held.addresses() == [t.data_ptr() for t in ts]


@pytest.mark.parametrize("i,new", [
    (0, torch.zeros(6, dtype=torch.bfloat16)), (0, torch.zeros(6, dtype=torch.int32)), (0, torch.zeros(5)),
    (0, torch.zeros(12)[::2]), (1, torch.zeros((4, 3), dtype=torch.bfloat16).t()), (2, torch.zeros(1)),
    (3, torch.zeros((), dtype=torch.float64)),
], ids=["type", "type of the same width", "size", "strided", "transposed", "no longer empty", "one value"])
def test_other_changes_are_refused(i, new):
    ts = tensors()
    held = gb._Tensors(ts)
    ts[i].data = new
    for _ in range(2):      # a second call as well
        with pytest.raises(ValueError, match=f"tensor {i} of the list has changed"):
            held.addresses()


def test_a_type_changed_in_place_at_the_same_address():
    t = torch.zeros(8)
    held = gb._Tensors([t])
    t.data = t.data.view(torch.bfloat16)[:8]
    assert t.data_ptr() == held.tensors[0].data_ptr()
    with pytest.raises(ValueError, match="has changed"):
        held.addresses()


def test_a_module_that_changes_its_type():
    """module.bfloat16() replaces the memory of the gradient tensors it has."""
    m = torch.nn.Linear(3, 5)
    m(torch.ones(2, 3)).sum().backward()
    grads = [p.grad for p in m.parameters()]
    held = gb._Tensors(grads)
    m.bfloat16()
    assert grads[0] is m.weight.grad and grads[0].dtype == torch.bfloat16
    with pytest.raises(ValueError, match="tensor 0 of the list has changed"):
        held.addresses()
