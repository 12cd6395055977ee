"""Refusals of the operators around the convolutions, on the host: every
invalid call is turned away before the first HIP call, by the binding or by
the C ABI, so these run without a GPU.
"""
import ctypes
import re
import time

import pytest
import torch

from backward_implicit_gemm_amd import binding as gb

FAKE = 0x10000     # never dereferenced: every call below fails validation
BAD, SMALL = gb.GC_ERR_INVALID_ARG, gb.GC_ERR_WORKSPACE
BIG = 1 << 40


# ------------------------------------------------------------------ the C ABI --
def embed_desc(rows=4, tokens=3, V=10, D=8, itype=gb.GC_I32, ld=None, ld_tok=None):
    return gb.gc_embed_desc(rows, tokens, V, D, itype, tokens * D if ld is None else ld,
                            tokens if ld_tok is None else ld_tok)


def embed_bwd(d, tok=FAKE, dout=FAKE, dtable=FAKE, ws=FAKE, n=BIG, dtype=0):
    return gb.lib().gc_embed_bwd(tok, dout, dtable, ws, n, ctypes.byref(d), 1.0, dtype, None)


def embed_fwd(d, tok=FAKE, table=FAKE, out=FAKE, dtype=0):
    return gb.lib().gc_embed_fwd(tok, table, out, ctypes.byref(d), 1.0, dtype, None)


@pytest.mark.parametrize("change", [
    dict(rows=-1), dict(tokens=-1), dict(V=0), dict(D=0), dict(itype=3), dict(itype=-1), dict(ld=23),
    dict(ld_tok=2), dict(rows=1 << 30, tokens=4), dict(tokens=1 << 20, D=1 << 20), dict(rows=1 << 20, ld=1 << 50),
])
def test_embed_descriptors(change):
    d = embed_desc(**change)
    assert embed_fwd(d) == BAD and embed_bwd(d) == BAD
    assert gb.lib().gc_embed_workspace_bytes(ctypes.byref(d), 0) == 0


def test_embed_pointers_types_and_workspace():
    d = embed_desc()
    L = gb.lib()
    assert L.gc_embed_fwd(FAKE, FAKE, FAKE, None, 1.0, 0, None) == BAD
    for name in ("tok", "table", "out"):
        assert embed_fwd(d, **{name: None}) == BAD
        assert embed_fwd(d, **{name: FAKE + 1}) == BAD
    for name in ("tok", "dout", "dtable"):
        assert embed_bwd(d, **{name: None}) == BAD
        assert embed_bwd(d, **{name: FAKE + 2}) == BAD
    assert embed_bwd(embed_desc(itype=gb.GC_I64), tok=FAKE + 4) == BAD
    assert embed_fwd(d, dtype=2) == BAD and embed_bwd(d, dtype=-1) == BAD
    need = L.gc_embed_workspace_bytes(ctypes.byref(d), 0)
    assert need > 0
    assert embed_bwd(d, ws=None) == SMALL and embed_bwd(d, n=need - 1) == SMALL and embed_bwd(d, ws=FAKE + 16) == SMALL
    assert L.gc_embed_workspace_bytes(ctypes.byref(d), 9) == 0


def norm_desc(B=2, C=12, H=3, W=4, groups=3, layout=0, act=1, eps=1e-5):
    return gb.gc_norm_desc(B, C, H, W, groups, layout, act, eps)


def norm_fwd(d, ws=FAKE, n=BIG, dtype=0, pt=0, **p):
    a = dict(x=FAKE, gamma=FAKE, beta=FAKE, y=FAKE, mean=FAKE, rstd=FAKE) | p
    return gb.lib().gc_group_norm_fwd(*a.values(), ws, n, ctypes.byref(d), dtype, pt, None)


def norm_bwd(d, ws=FAKE, n=BIG, dtype=0, pt=0, **p):
    a = dict(x=FAKE, gamma=FAKE, beta=FAKE, dy=FAKE, mean=FAKE, rstd=FAKE, dx=FAKE, dgamma=FAKE, dbeta=FAKE) | p
    return gb.lib().gc_group_norm_bwd(*a.values(), ws, n, ctypes.byref(d), dtype, pt, None)


@pytest.mark.parametrize("change", [
    dict(B=0), dict(C=0), dict(H=0), dict(W=-1), dict(groups=0), dict(groups=5), dict(groups=24), dict(layout=2),
    dict(act=4), dict(act=-1), dict(eps=-1e-9), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(H=1 << 16, W=1 << 16), dict(C=1 << 12, groups=1, H=1 << 10, W=1 << 10),
    dict(B=(1 << 30) + 1), dict(H=1, W=(1 << 30) + 1, C=1, groups=1), dict(C=(1 << 23) + 1, groups=1, H=1, W=1),
])
def test_norm_descriptors(change):
    d = norm_desc(**change)
    assert norm_fwd(d) == BAD and norm_bwd(d) == BAD
    for op in (gb.GC_OP_FWD, gb.GC_OP_BWD):
        assert gb.lib().gc_group_norm_workspace_bytes(op, ctypes.byref(d), 0) == 0


def test_norm_pointers_types_and_workspace():
    d = norm_desc()
    for name in ("x", "y"):
        assert norm_fwd(d, **{name: None}) == BAD
    for name in ("x", "gamma", "beta", "y", "mean", "rstd"):
        assert norm_fwd(d, **{name: FAKE + 2}) == BAD
    for name in ("x", "dy", "mean", "rstd", "dx"):
        assert norm_bwd(d, **{name: None}) == BAD
    for name in ("x", "gamma", "beta", "dy", "mean", "rstd", "dx", "dgamma", "dbeta"):
        assert norm_bwd(d, **{name: FAKE + 2}) == BAD
    assert norm_fwd(d, dtype=2) == BAD and norm_fwd(d, dtype=gb.GC_F32, pt=gb.GC_BF16) == BAD
    assert norm_bwd(d, dtype=2) == BAD and norm_bwd(d, dtype=gb.GC_F32, pt=gb.GC_BF16) == BAD
    L = gb.lib()
    assert L.gc_group_norm_workspace_bytes(gb.GC_OP_BWD_DATA, ctypes.byref(d), 0) == 0
    for op, call in ((gb.GC_OP_FWD, norm_fwd), (gb.GC_OP_BWD, norm_bwd)):
        big = norm_desc(C=64, groups=1, H=300, W=300)     # one group of 5.8 million elements
        need = L.gc_group_norm_workspace_bytes(op, ctypes.byref(big), 0)
        assert need > 0
        assert call(big, ws=None, n=0) == SMALL and call(big, n=need - 1) == SMALL and call(big, ws=FAKE + 8) == SMALL


def clip(items, count=None, max_norm=1.0, prescale=1.0, eps=0.0, norm=FAKE, ws=FAKE, n=BIG):
    arr = (gb.gc_tensor * max(1, len(items)))(*[gb.gc_tensor(*i) for i in items])
    return gb.lib().gc_grad_clip(arr, len(items) if count is None else count, max_norm, prescale, eps, norm, ws, n, None)


def test_clip_arguments():
    good = (FAKE, FAKE, 5, gb.GC_F32)
    nan, inf = float("nan"), float("inf")
    L = gb.lib()
    assert L.gc_grad_clip(None, 1, 1.0, 1.0, 0.0, FAKE, FAKE, BIG, None) == BAD
    for bad in ((None, FAKE, 5, 0), (FAKE, None, 5, 0), (FAKE, FAKE, -1, 0), (FAKE, FAKE, 5, 2),
                (FAKE + 2, FAKE, 5, 0), (FAKE, FAKE + 1, 5, 1), (FAKE, FAKE, 1 << 43, 0)):
        assert clip([good, bad]) == BAD
    for kw in (dict(max_norm=-1.0), dict(max_norm=nan), dict(prescale=nan), dict(prescale=inf), dict(eps=-1.0),
               dict(eps=nan), dict(norm=None), dict(norm=FAKE + 1), dict(count=-1)):
        assert clip([good], **kw) == BAD
    need = L.gc_grad_clip_workspace_bytes(1)
    assert clip([good], ws=None) == SMALL and clip([good], n=need - 1) == SMALL and clip([good], ws=FAKE + 8) == SMALL
    assert L.gc_grad_norm(None, 0, 1.0, None, FAKE, BIG, None) == BAD
    assert L.gc_grad_clip_workspace_bytes(-1) == 0
    assert L.gc_grad_clip_workspace_bytes(1000) > L.gc_grad_clip_workspace_bytes(96) == need


# ----------------------------------------------------------------- the binding --
def test_binding_embedding_refusals():
    e = gb.Embedding(2, 3, 10, 4, torch.float32, device="cpu")
    tok, table, out = torch.zeros((2, 3), dtype=torch.int32), torch.zeros((10, 4)), torch.zeros((2, 3, 4))
    with pytest.raises(ValueError, match="tokens has shape"):
        e.fwd(tok[:1], table, out)
    with pytest.raises(TypeError, match="tokens has dtype"):
        e.fwd(tok.float(), table, out)
    with pytest.raises(ValueError, match="out has shape"):
        e.fwd(tok, table, out[:, :2])
    with pytest.raises(TypeError, match="out has dtype"):
        e.fwd(tok, table, out.bfloat16())
    with pytest.raises(ValueError, match="dense within a row"):
        e.fwd(tok, table, torch.zeros((2, 4, 3)).transpose(1, 2))
    with pytest.raises(ValueError, match="must not overlap"):
        e.fwd(tok, table, torch.zeros(24).as_strided((2, 3, 4), (8, 4, 1)))
    with pytest.raises(ValueError, match="must not overlap"):
        e.bwd(tok[:1].expand(2, 3), out, table)
    with pytest.raises(ValueError, match="table has shape"):
        e.fwd(tok, table[:9], out)
    with pytest.raises(TypeError, match="table has dtype"):
        e.fwd(tok, table.bfloat16(), out)
    with pytest.raises(ValueError, match="device tensor"):
        e.fwd(tok, table, out)
    with pytest.raises(TypeError, match="unsupported dtype"):
        gb.Embedding(2, 3, 10, 4, torch.float16, device="cpu")


def test_binding_norm_refusals():
    gn = gb.GroupNorm((2, 8, 3, 4), 2, "relu", torch.float32, "nhwc", device="cpu")
    x = torch.zeros((2, 8, 3, 4)).contiguous(memory_format=torch.channels_last)
    p, m = torch.zeros(8), torch.zeros((2, 2))
    with pytest.raises(ValueError, match="x has shape"):
        gn.fwd(x[:1], p, p, x)
    with pytest.raises(ValueError, match="x must be dense"):
        gn.fwd(x.contiguous(), p, p, x)
    with pytest.raises(TypeError, match="x has dtype"):
        gn.fwd(x.bfloat16(), p, p, x)
    with pytest.raises(ValueError, match="device tensor"):
        gn.bwd(x, p, p, x, m, m, x)
    with pytest.raises(ValueError, match="unknown act"):
        gb.GroupNorm((2, 8, 3, 4), 2, "tanh", torch.float32, device="cpu")
    with pytest.raises(ValueError, match="unknown layout"):
        gb.GroupNorm((2, 8, 3, 4), 2, "relu", torch.float32, "chwn", device="cpu")
    with pytest.raises(TypeError, match="param_dtype"):
        gb.GroupNorm((2, 8, 3, 4), 2, "relu", torch.float32, param_dtype=torch.bfloat16, device="cpu")


def test_binding_clip_refusals():
    g = torch.zeros(6)
    with pytest.raises(ValueError, match="device tensors"):
        gb.GradClip([g])
    with pytest.raises(ValueError, match="outputs"):
        gb.GradClip([g], [])
    with pytest.raises(ValueError, match="elements of"):
        gb.GradClip([g], [g[:5]])
    with pytest.raises(ValueError, match="elements of"):
        gb.GradClip([g], [g.bfloat16()])
    with pytest.raises(ValueError, match="contiguous"):
        gb.GradClip([torch.zeros((3, 4)).t()])


def test_binding_refuses_invalid_descriptors():
    """A shape that the C ABI refuses is refused when the helper is made."""
    with pytest.raises(ValueError):
        gb.GroupNorm((2, 8, 3, 4), 3, "relu", torch.float32, device="cpu")
    with pytest.raises(ValueError):
        gb.Embedding(2, 3, 0, 4, torch.float32, device="cpu")


# ------------------------------------------------------------------- the plans --
def norm_plan(op, shape, groups, layout, dtype):
    B, C, H, W = shape
    return gb.gc_group_norm_plan_name(op, gb.gc_norm_desc(B, C, H, W, groups, layout, 0, 1e-5), dtype)


@pytest.mark.parametrize("op", [gb.GC_OP_FWD, gb.GC_OP_BWD])
@pytest.mark.parametrize("dtype", [gb.GC_F32, gb.GC_BF16])
@pytest.mark.parametrize("layout", [gb.GC_NCHW, gb.GC_NHWC])
def test_the_policy_layers_stay_resident(op, dtype, layout):
    for B in (1, 37, 256, 1024, 16384, 32768):
        for shape, groups in (((B, 128, 3, 4), 8), ((B, 128, 1, 2), 16), ((B, 59, 11, 15), 1)):
            assert norm_plan(op, shape, groups, layout, dtype).startswith("res_"), (shape, groups)


def test_large_groups_are_split():
    for layout in (gb.GC_NCHW, gb.GC_NHWC):
        for op in (gb.GC_OP_FWD, gb.GC_OP_BWD):
            assert norm_plan(op, (2, 64, 300, 300), 1, layout, gb.GC_BF16).startswith("norm_split")


def test_plans_of_extreme_shapes():
    """The most images, channels, groups and positions: grids and workspaces without overflow, found without a walk."""
    most, wide = 2 ** 30, 2 ** 23
    for shape, groups in (((1, wide, 1, 1), wide), ((1, wide, 1, 1), 1), ((1, 1, 1, most), 1), ((1, wide, 1, 1), wide // 2),
                          ((most, 1, 1, 1), 1), ((most, 8, 16, 16), 8), ((1, wide, 1, 2), 1), ((most, 64, 1, 2), 8),
                          ((3, 7, 1, most // 7), 7), ((most, 512, 3, 4), 1), ((2 ** 20, wide, 8, 16), 1)):
        for layout in (gb.GC_NCHW, gb.GC_NHWC):
            for dtype in (gb.GC_F32, gb.GC_BF16):
                for op in (gb.GC_OP_FWD, gb.GC_OP_BWD):
                    start = time.monotonic()
                    name = norm_plan(op, shape, groups, layout, dtype)
                    d = gb.gc_norm_desc(*shape, groups, layout, 0, 1e-5)
                    need = gb.lib().gc_group_norm_workspace_bytes(op, ctypes.byref(d), dtype)
                    assert time.monotonic() - start < 0.5, (shape, groups)
                    assert need < 2 ** 45, (shape, groups, need)
                    numbers = [int(v) for v in re.findall(r"(?:grid|chunks)=(-?[0-9]+)", name)]
                    assert name == "none" or (numbers and min(numbers) >= 1 and max(numbers) < 2 ** 31), name


def test_embedding_plans():
    """Few cells (padded rows x 32-column slabs x tokens) are a one-hot product, others are sorted."""
    for n, V, D, dtype, name in ((48128, 128, 32, 0, "onehot"), (1540096, 128, 32, 1, "onehot"), (12, 1024, 2, 0, "onehot"),
                                 (12, 4000, 32, 1, "onehot"), (12, 4097, 32, 1, "sort"), (12, 4000, 32, 0, "sort"),
                                 (400000, 512, 32, 0, "sort"), (400000, 512, 32, 1, "onehot"),
                                 (12, 128, 1, 1, "sort"), (32768, 40960, 1024, 1, "sort")):
        d = embed_desc(rows=n, tokens=1, V=V, D=D)
        assert gb.gc_embed_plan_name(d, dtype) == "embed_grad_" + name, (n, V, D, dtype)
    assert gb.gc_embed_plan_name(embed_desc(rows=0), gb.GC_F32) == "embed_grad_sort"


def test_plan_name_errors():
    d, L = norm_desc(), gb.lib()
    buf = ctypes.create_string_buffer(16)
    assert L.gc_group_norm_plan_name(gb.GC_OP_FWD, ctypes.byref(d), 0, None, 16) == BAD
    assert L.gc_group_norm_plan_name(gb.GC_OP_FWD, ctypes.byref(d), 0, buf, 0) == BAD
    assert L.gc_group_norm_plan_name(gb.GC_OP_BWD_BIAS, ctypes.byref(d), 0, buf, 16) == BAD
    assert L.gc_group_norm_plan_name(gb.GC_OP_FWD, ctypes.byref(d), 5, buf, 16) == BAD
    assert L.gc_embed_plan_name(ctypes.byref(embed_desc(V=0)), 0, buf, 16) == BAD
    assert L.gc_embed_plan_name(ctypes.byref(embed_desc()), 0, None, 16) == BAD
    assert L.gc_group_norm_plan_name(gb.GC_OP_FWD, ctypes.byref(d), 0, buf, 16) == gb.GC_OK
    assert len(buf.value) == 15        # truncated, with its end
