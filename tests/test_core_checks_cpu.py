"""The remembered checks of the recurrent core's calls, on the host: a call like the last one is not
checked in full again, also in place, and any other one is."""
import pytest
import torch

from backward_implicit_gemm_amd import binding as gb


class Counted:
    """Stands for a helper's full check: counts its calls."""

    def __init__(self, keep=True):
        self.calls, self.keep = 0, keep

    def __call__(self, helper, *tensors):
        self.calls += 1
        return f"desc {self.calls}", self.keep


def tensors(n, *shape):
    return [torch.zeros(shape or (3, 4)) for _ in range(n)]


# which places of a call hold the same tensor, None for one left out
PATTERNS = [
    (0, 1, 2), (0, 0, 1), (0, 1, 0), (0, 1, 1), (0, 0, 0), (0, None, 0), (None, 0, 0),
    (0, 1, None, None, 0, 2),        # a state as h0 and as last
    (0, 1, 2, 3, 4, 1, None, 5),     # the stream as residual and as total
    (0, 0, 1, 1, 2, 2),
]


@pytest.mark.parametrize("pattern", PATTERNS, ids=str)
def test_a_call_like_the_last_is_not_checked_again(pattern):
    full = Counted()
    check = gb._Checked(full)

    def call(ts):
        return check(None, *(None if k is None else ts[k] for k in pattern))

    first = call(tensors(6))
    for _ in range(3):
        ts = tensors(6)              # other tensors of the same kind
        desc, at = call(ts)
        assert desc == first[0]
        assert at == [None if k is None else ts[k].data_ptr() for k in pattern]
    assert full.calls == 1


@pytest.mark.parametrize("first", PATTERNS[:7], ids=str)
@pytest.mark.parametrize("then", PATTERNS[:7], ids=str)
def test_other_tensors_as_one_are_checked(first, then):
    full = Counted()
    check = gb._Checked(full)
    for pattern in (first, then, first):
        ts = tensors(3)
        check(None, *(None if k is None else ts[k] for k in pattern))
    assert full.calls == (1 if first == then else 3)


@pytest.mark.parametrize("change", [lambda t: t.double(), lambda t: t[:2], lambda t: t.t(), lambda t: t[:, ::2],
                                    lambda t: torch.empty((3, 8))[:, :4]])
@pytest.mark.parametrize("place", range(4))
def test_another_kind_of_tensor_is_checked(place, change):
    full = Counted()
    check = gb._Checked(full)
    a, b, c = tensors(3)
    check(None, a, b, a, c)
    args = [a, b, a, c]
    args[place] = change(args[place])
    check(None, *args)
    assert full.calls == 2
    check(None, *args)
    assert full.calls == 2


def test_what_must_not_be_remembered_is_checked_each_time():
    full = Counted(keep=False)
    check = gb._Checked(full)
    a, b = tensors(2)
    for _ in range(3):
        check(None, a, b)
    assert full.calls == 3


def test_a_failed_check_is_not_remembered():
    def full(helper, *ts):
        if ts[0].shape != (3, 4):
            raise ValueError("shape")
        return "desc", True

    check = gb._Checked(full)
    good, bad = torch.zeros(3, 4), torch.zeros(2, 4)
    check(None, good, good)
    for _ in range(2):
        with pytest.raises(ValueError):
            check(None, bad, bad)
    assert check(None, good, good)[0] == "desc"


@pytest.mark.parametrize("other", [lambda t: t, lambda t: t[:2]], ids=["kept", "refused"])
def test_another_threads_call_in_between(other):
    """A call whose comparison is under way when another one replaces what is remembered, or drops it."""
    full = Counted()
    check = gb._Checked(full)
    a, b = tensors(2)
    desc, _ = check(None, a, b)
    remembered = check.last

    def compare(*ts):
        full.keep = other(a) is a
        check(None, other(b), None)
        return True

    check.last = (*remembered[:-1], compare)
    assert check(None, a, b) == (desc, [a.data_ptr(), b.data_ptr()])
