"""Refusals of the recurrent core's operators, on the host: every invalid call is turned
away before the first HIP call, by the binding or by the C ABI, so these run without
a GPU.
"""
import ctypes
import re

import pytest
import torch

from backward_implicit_gemm_amd import binding as gb

FAKE = 0x10000     # never dereferenced: every call below fails validation
BAD, SMALL, UNSUPPORTED = gb.GC_ERR_INVALID_ARG, gb.GC_ERR_WORKSPACE, gb.GC_ERR_UNSUPPORTED
BIG = 1 << 44
NAN, INF = float("nan"), float("inf")


# ------------------------------------------------------------------ the C ABI --
def rows_desc(rows=4, D=24, eps=1e-5, **ld):
    d = gb.gc_layer_norm_desc(rows, D, eps, D, D, D, D)
    for k, v in ld.items():
        setattr(d, k, v)
    return d


def rows_fwd(d, dtype=0, pt=0, **p):
    a = dict(x=FAKE, residual=FAKE, gamma=FAKE, beta=FAKE, y=FAKE, total=FAKE, mean=FAKE, rstd=FAKE) | p
    return gb.lib().gc_layer_norm_fwd(*a.values(), d if d is None else ctypes.byref(d), dtype, pt, None)


def rows_bwd(d, dtype=0, pt=0, ws=FAKE, n=BIG, **p):
    a = dict(x=FAKE, gamma=FAKE, dy=FAKE, dtotal=FAKE, mean=FAKE, rstd=FAKE, dx=FAKE, dgamma=FAKE, dbeta=FAKE) | p
    return gb.lib().gc_layer_norm_bwd(*a.values(), ws, n, d if d is None else ctypes.byref(d), dtype, pt, None)


@pytest.mark.parametrize("change", [
    dict(rows=-1), dict(rows=1 << 31), dict(D=0), dict(D=-3), dict(D=(1 << 23) + 1), dict(eps=-1e-9), dict(eps=NAN),
    dict(eps=INF), dict(ld_x=23), dict(ld_y=0), dict(ld_total=-24), dict(ld_residual=23), dict(ld_y=1 << 60),
])
def test_layer_norm_descriptors(change):
    d = rows_desc(**change)
    assert rows_fwd(d) == BAD and rows_bwd(d) == BAD
    assert gb.lib().gc_layer_norm_workspace_bytes(ctypes.byref(d), 0) == 0


def test_layer_norm_pointers_types_and_workspace():
    d = rows_desc()
    assert rows_fwd(None) == BAD and rows_bwd(None) == BAD
    for name in ("x", "y"):
        assert rows_fwd(d, **{name: None}) == BAD
    for name in ("x", "residual", "gamma", "beta", "y", "total", "mean", "rstd"):
        assert rows_fwd(d, **{name: FAKE + 2}) == BAD
    for name in ("x", "dy", "mean", "rstd", "dx"):
        assert rows_bwd(d, **{name: None}) == BAD
    for name in ("x", "gamma", "dy", "dtotal", "mean", "rstd", "dx", "dgamma", "dbeta"):
        assert rows_bwd(d, **{name: FAKE + 2}) == BAD
    for call in (rows_fwd, rows_bwd):
        assert call(d, dtype=2) == BAD and call(d, dtype=gb.GC_F32, pt=gb.GC_BF16) == BAD and call(d, pt=7) == BAD
    need = gb.lib().gc_layer_norm_workspace_bytes(ctypes.byref(d), 0)
    assert need > 0 and gb.lib().gc_layer_norm_workspace_bytes(ctypes.byref(d), 5) == 0
    assert rows_bwd(d, ws=None) == SMALL and rows_bwd(d, n=need - 1) == SMALL and rows_bwd(d, ws=FAKE + 8) == SMALL
    # without rows there is nothing to do in the forward
    assert rows_fwd(rows_desc(rows=0), x=None, y=None) == gb.GC_OK


DENSE = dict(gate=(70, 7), value=(70, 7), out=(70, 7), dgate=(70, 7), dvalue=(70, 7), reset=(10, 1))


def scan_desc(B=3, T=10, D=7, coupled=1, **strides):
    s = DENSE | strides
    return gb.gc_recurrence_desc(B, T, D, coupled, *(gb.gc_strides(*s[k]) for k in DENSE))


def scan_fwd(d, dtype=0, ws=FAKE, n=BIG, **p):
    a = dict(gate=FAKE, value=FAKE, h0=FAKE, reset=FAKE, lengths=FAKE, out=FAKE, last=FAKE, states=FAKE) | p
    return gb.lib().gc_recurrence_fwd(*a.values(), ws, n, d if d is None else ctypes.byref(d), dtype, None)


def scan_bwd(d, dtype=0, ws=FAKE, n=BIG, **p):
    a = dict(gate=FAKE, value=FAKE, states=FAKE, reset=FAKE, lengths=FAKE, dout=FAKE, dlast=FAKE, dgate=FAKE, dvalue=FAKE,
             dh0=FAKE) | p
    return gb.lib().gc_recurrence_bwd(*a.values(), ws, n, d if d is None else ctypes.byref(d), dtype, None)


@pytest.mark.parametrize("change", [
    dict(B=-1), dict(T=-1), dict(T=(1 << 30) + 1), dict(D=0), dict(coupled=2), dict(coupled=-1), dict(gate=(-1, 7)),
    dict(value=(70, -7)), dict(reset=(-1, 1)), dict(gate=(1 << 60, 7)), dict(reset=(1, 1 << 58)),
])
def test_recurrence_descriptors(change):
    d = scan_desc(**change)
    assert scan_fwd(d) == BAD and scan_bwd(d) == BAD
    for op in (gb.GC_OP_FWD, gb.GC_OP_BWD):
        assert gb.lib().gc_recurrence_workspace_bytes(op, ctypes.byref(d), 0) == 0


@pytest.mark.parametrize("strides", [(69, 7), (70, 6), (7, 20), (0, 7), (70, 0), (7, 7)])
def test_recurrence_outputs_do_not_overlap(strides):
    assert scan_fwd(scan_desc(out=strides)) == BAD
    assert scan_bwd(scan_desc(dgate=strides)) == BAD and scan_bwd(scan_desc(dvalue=strides)) == BAD


def test_recurrence_pointers_types_and_workspace():
    d = scan_desc()
    assert scan_fwd(None) == BAD and scan_bwd(None) == BAD
    for name in ("gate", "value", "out"):
        assert scan_fwd(d, **{name: None}) == BAD
    for name in ("gate", "value", "out", "h0", "last", "states", "lengths"):
        assert scan_fwd(d, **{name: FAKE + 2}) == BAD
    for name in ("gate", "value", "states", "dout", "dgate", "dvalue"):
        assert scan_bwd(d, **{name: None}) == BAD
    for name in ("gate", "value", "states", "dout", "dgate", "dvalue", "dlast", "dh0", "lengths"):
        assert scan_bwd(d, **{name: FAKE + 2}) == BAD
    assert scan_fwd(d, dtype=2) == BAD and scan_bwd(d, dtype=-1) == BAD
    L = gb.lib()
    wide = (1 << 20, 1 << 10)
    d = scan_desc(B=1, T=100000, D=8, **{k: wide for k in DENSE})
    for op, call in ((gb.GC_OP_FWD, scan_fwd), (gb.GC_OP_BWD, scan_bwd)):
        need = L.gc_recurrence_workspace_bytes(op, ctypes.byref(d), 0)
        assert need > 0 and L.gc_recurrence_workspace_bytes(op, ctypes.byref(d), 3) == 0
        assert call(d, ws=None) == SMALL and call(d, n=need - 1) == SMALL and call(d, ws=FAKE + 64) == SMALL
    assert L.gc_recurrence_workspace_bytes(gb.GC_OP_BWD_DATA, ctypes.byref(d), 0) == 0
    far = scan_desc(B=1 << 20, T=1, D=1 << 12, **{k: (1 << 12, 1 << 12) for k in DENSE})
    assert scan_fwd(far) == UNSUPPORTED and scan_bwd(far) == UNSUPPORTED
    # no sequences: nothing to do
    assert scan_fwd(scan_desc(B=0), gate=None, value=None, out=None, h0=None, last=None) == gb.GC_OK


def distill_desc(rows=5, V=30, K=4, itype=gb.GC_I32, teacher=gb.GC_F32, t=1.0, ld=30, ld_grad=30, ld_index=4, ld_teacher=4):
    return gb.gc_distill_desc(rows, V, K, itype, teacher, t, ld, ld_grad, ld_index, ld_teacher)


def distill_calls(d, dtype=0, **p):
    a = dict(logits=FAKE, index=FAKE, teacher=FAKE, loss=FAKE, peak=FAKE, mass=FAKE, dloss=FAKE, dlogits=FAKE) | p
    L, r = gb.lib(), d if d is None else ctypes.byref(d)
    first = a["logits"], a["index"], a["teacher"]
    return (L.gc_distill_fwd(*first, a["loss"], a["peak"], a["mass"], r, dtype, None),
            L.gc_distill_bwd(*first, a["peak"], a["mass"], a["dloss"], a["dlogits"], r, dtype, None),
            L.gc_distill_step(*first, a["dloss"], a["loss"], a["dlogits"], r, dtype, None))


@pytest.mark.parametrize("change", [
    dict(rows=-1), dict(rows=1 << 31), dict(V=0), dict(K=0), dict(K=1025, ld_index=1025, ld_teacher=1025), dict(itype=gb.GC_U8),
    dict(itype=-1), dict(teacher=2), dict(t=0.0), dict(t=-1.0), dict(t=NAN), dict(t=INF), dict(t=9e-19), dict(t=1.1e18), dict(ld=29), dict(ld_grad=29),
    dict(ld_index=3), dict(ld_teacher=3), dict(ld=1 << 59),
])
def test_distill_descriptors(change):
    assert distill_calls(distill_desc(**change)) == (BAD,) * 3


def test_distill_pointers_and_types():
    d = distill_desc()
    assert distill_calls(None) == (BAD,) * 3 and distill_calls(d, dtype=2) == (BAD,) * 3
    for name in ("logits", "index", "teacher"):
        assert distill_calls(d, **{name: None}) == (BAD,) * 3
        assert distill_calls(d, **{name: FAKE + 2}) == (BAD,) * 3
    assert distill_calls(distill_desc(itype=gb.GC_I64), index=FAKE + 4) == (BAD,) * 3
    all_bad = dict(loss=FAKE + 2, dloss=FAKE + 2)
    assert distill_calls(d, **all_bad) == (BAD,) * 3
    assert distill_calls(d, loss=None, dloss=None) == (BAD,) * 3
    assert distill_calls(d, loss=FAKE + 1, peak=None, dlogits=None) == (BAD,) * 3
    assert distill_calls(d, loss=FAKE + 1, mass=FAKE + 1, dlogits=FAKE + 1) == (BAD,) * 3
    assert distill_calls(distill_desc(rows=0)) == (gb.GC_OK,) * 3
    many = distill_desc(rows=1 << 30, V=1 << 20, ld=1 << 20, ld_grad=1 << 20)
    assert distill_calls(many) == (UNSUPPORTED,) * 3


# ----------------------------------------------------------------- the binding --
def test_binding_layer_norm_refusals():
    n = gb.LayerNorm(3, 8, torch.float32, device="cpu")
    x, p, s = torch.zeros((3, 8)), torch.zeros(8), torch.zeros(3)
    for call, match in ((lambda: n.fwd(x[:2], p, p, x), "x has shape"), (lambda: n.fwd(x, p[:7], p, x), "device tensor"),
                        (lambda: n.fwd(torch.zeros((8, 3)).t(), p, p, x), "dense within a row"),
                        (lambda: n.fwd(x[:1].expand(3, 8), p, p, x), "must not overlap"),
                        (lambda: n.fwd(x, p, p, x), "device tensor"),
                        (lambda: n.bwd(x, p, x[:, :7], s, s, x), "device tensor")):
        with pytest.raises(ValueError, match=match):
            call()
    with pytest.raises(TypeError, match="x has dtype"):
        n.fwd(x.bfloat16(), p, p, x)
    with pytest.raises(TypeError, match="param_dtype"):
        gb.LayerNorm(3, 8, torch.float32, param_dtype=torch.bfloat16, device="cpu")
    with pytest.raises(TypeError, match="unsupported dtype"):
        gb.LayerNorm(3, 8, torch.float16, device="cpu")
    for rows, dim, eps in ((-1, 8, 0.0), (1 << 31, 8, 0.0), (3, 0, 0.0), (3, (1 << 23) + 1, 0.0), (3, 8, -1.0), (3, 8, NAN),
                           (3, 8, 1e39)):
        with pytest.raises(ValueError):
            gb.LayerNorm(rows, dim, torch.float32, eps, device="cpu")


def test_binding_recurrence_refusals():
    r = gb.Recurrence(2, 5, 4, torch.float32, device="cpu")
    x = torch.zeros((2, 5, 4))
    for call, match in ((lambda: r.fwd(x[:1], x, x), "gate has shape"), (lambda: r.fwd(x, x, x), "device tensor"),
                        (lambda: r.fwd(torch.zeros((2, 4, 5)).transpose(1, 2), x, x), "channels of gate"),):
        with pytest.raises(ValueError, match=match):
            call()
    with pytest.raises(TypeError, match="gate has dtype"):
        r.fwd(x.bfloat16(), x, x)
    for B, T, D in ((-1, 5, 4), (2, -1, 4), (2, (1 << 30) + 1, 4), (2, 5, 0), (1 << 31, 1, 1)):
        with pytest.raises(ValueError):
            gb.Recurrence(B, T, D, torch.float32, device="cpu")
    assert r.states_shape == (2, 1, 4) and gb.Recurrence(2, 17, 4, torch.float32, device="cpu").states_shape == (2, 2, 4)
    assert gb.Recurrence(2, 0, 4, torch.float32, device="cpu").states_shape == (2, 0, 4)
    for strides in ((20, 4), (4, 8), (100, 9)):
        assert r._apart(*strides)
    for strides in ((19, 4), (20, 3), (4, 7), (0, 4), (20, 0)):
        assert not r._apart(*strides)


def test_binding_distill_refusals():
    h = gb.Distill(3, 9, 2, torch.float32, device="cpu")
    z, i, t, row = torch.zeros((3, 9)), torch.zeros((3, 2), dtype=torch.int32), torch.zeros((3, 2)), torch.zeros(3)
    with pytest.raises(TypeError, match="index has dtype"):
        h.fwd(z, i.float(), t, row)
    with pytest.raises(ValueError, match="logits has shape"):
        h.fwd(z[:, :8], i, t, row)
    with pytest.raises(ValueError, match="device tensor"):
        h.fwd(z, i, t, row)
    for args in ((-1, 9, 2), (3, 0, 2), (3, 9, 0), (3, 9, 1025), (1 << 31, 9, 2)):
        with pytest.raises(ValueError):
            gb.Distill(*args, torch.float32, device="cpu")
    for t in (0.0, -1.0, NAN, INF, 1e-60, 1e60, 9e-19, 1.1e18):
        with pytest.raises(ValueError, match="temperature"):
            gb.Distill(3, 9, 2, torch.float32, t, device="cpu")
    with pytest.raises(TypeError, match="unsupported dtype"):
        gb.Distill(3, 9, 2, torch.float32, teacher_dtype=torch.float16, device="cpu")


def test_launches_go_to_the_tensors_device(monkeypatch):
    """With another device current, the call is made with the helper's, which is put back."""
    current = [0]

    class Switch:
        def __init__(self, device):
            self.index = device.index

        def __enter__(self):
            self.was, current[0] = current[0], self.index

        def __exit__(self, *_):
            current[0] = self.was

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    monkeypatch.setattr(torch.cuda, "device", Switch)
    for index in (0, 1):
        assert gb._launch(torch.device("cuda", index), lambda a: (a, current[0]), 7) == (7, index)
        assert current[0] == 0


# ------------------------------------------------------------------- the plans --
def numbers(name):
    return [int(v) for v in re.findall(r"(?:grid|chunks|steps|lanes|team|threads|NV?)=(-?[0-9]+)", name)]


def test_plans_of_extreme_shapes():
    most = 2 ** 31 - 1
    for dtype in (gb.GC_F32, gb.GC_BF16):
        for op in (gb.GC_OP_FWD, gb.GC_OP_BWD):
            for rows, D in ((1, 1), (most, 1), (most, 1 << 23), (1, 1 << 23), (5, 7), (300, 16385)):
                d = rows_desc(rows, D)
                name = gb.gc_layer_norm_plan_name(op, d, dtype)
                assert min(numbers(name)) >= 1 and max(numbers(name)) < 2 ** 31, name
                assert gb.lib().gc_layer_norm_workspace_bytes(ctypes.byref(d), dtype) < 2 ** 36
            for B, T, D in ((1, 1, 1), (1, 1 << 30, 1), (most, 1, 1), (1, 1 << 20, most), (3, 17, 5), (1 << 15, 1 << 30, 1 << 15)):
                s = {k: (T * D, D) for k in DENSE}
                d = scan_desc(B, T, D, **s)
                name = gb.gc_recurrence_plan_name(op, d, dtype)
                found = numbers(name)
                assert min(found) >= 1 and max(found) < 2 ** 31, name
                chunks, steps = (int(re.search(f"{k}=([0-9]+)", name).group(1)) for k in ("chunks", "steps"))
                assert (chunks - 1) * steps < T <= chunks * steps and steps % 16 == 0, name
        for op in (gb.GC_OP_FWD, gb.GC_OP_BWD, gb.GC_OP_STEP):
            for rows, V, K in ((1, 1, 1), (1 << 20, 1, 1024), (1, most, 1024), (most, 1, 1), (7, 100000, 300), (3, 9, 1000)):
                name = gb.gc_distill_plan_name(op, distill_desc(rows, V, K, ld=V, ld_grad=V, ld_index=K, ld_teacher=K), dtype)
                assert "none" in name or 0 <= min(numbers(name)) and max(numbers(name)) < 2 ** 31, name


def test_plan_name_errors():
    L, buf = gb.lib(), ctypes.create_string_buffer(8)
    for fn, d in ((L.gc_layer_norm_plan_name, rows_desc()), (L.gc_recurrence_plan_name, scan_desc()),
                  (L.gc_distill_plan_name, distill_desc())):
        assert fn(gb.GC_OP_FWD, ctypes.byref(d), 0, buf, 8) == gb.GC_OK
        for bad in ((gb.GC_OP_BWD_DATA, ctypes.byref(d), 0, buf, 8), (gb.GC_OP_FWD, None, 0, buf, 8),
                    (gb.GC_OP_FWD, ctypes.byref(d), 4, buf, 8), (gb.GC_OP_FWD, ctypes.byref(d), 0, None, 8),
                    (gb.GC_OP_FWD, ctypes.byref(d), 0, buf, 0)):
            assert fn(*bad) == BAD


def test_recurrence_workspace_does_not_depend_on_distances():
    """A helper's workspace serves every layout its calls bring, sequences 4 GiB apart among them."""
    L = gb.lib()
    for dtype in (gb.GC_F32, gb.GC_BF16):
        for op in (gb.GC_OP_FWD, gb.GC_OP_BWD):
            for B, T, D in ((3, 300000, 10), (40, 1000, 33), (7, 12001, 777), (20, 300, 300), (1, 5000, 4096)):
                sizes = set()
                for batch, step in ((T * D, D), (D, B * D), (1 << 32, D), (D, 1 << 28), (1 << 40, 2 * D)):
                    d = scan_desc(B, T, D, **{k: (batch, step) for k in DENSE})
                    sizes.add(L.gc_recurrence_workspace_bytes(op, ctypes.byref(d), dtype))
                assert len(sizes) == 1 and min(sizes) > 0, (B, T, D, sizes)
