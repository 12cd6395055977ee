"""GPU: embedding lookup with scaling and its gradient against their
definitions in 64 bits.

Tokens are uniform, skewed (long runs of one value after sorting), all equal
or all empty; row lengths are odd, shorter than a vector and longer than a
workgroup; rows of out and dout lie apart.  The forward rounds a product
(2^-24) and the result; a gradient is a sum of m terms, off by at most
m * 2^-24 of its absolute terms, and rounded.
"""
import pytest
import torch

import train_ref as ref
from backward_implicit_gemm_amd import binding as gb
from parity import Guarded

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def setup_module():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    gb.lib()


def tokens(rows, T, V, kind, index, seed, extra=0):
    gen = torch.Generator("cuda").manual_seed(seed)
    u = torch.rand((rows, T + extra), generator=gen, device="cuda", dtype=torch.float64)
    power, empty = {"uniform": (1, 0.0), "skewed": (6, 0.1), "equal": (0, 0.0), "empty": (1, 1.0)}[kind]
    t = (u ** power * V).long().clamp(max=V - 1)
    if empty:
        out = torch.rand(t.shape, generator=gen, device="cuda") < empty
        t[out] = V + 5 if index == torch.uint8 else -1
        t[out & (u < 0.5)] = min(V, 255)
    return t.to(index)[:, :T]


def apart(rows, T, D, dtype, extra, offset=0, fill=None):
    """A (rows, T, D) view whose rows lie `extra` elements further apart, the guard of its buffer and the gaps."""
    g = Guarded((rows, T * D + extra), dtype, offset=offset)
    if fill is not None:
        g.t.copy_(fill)
    return g, g.t[:, :T * D].unflatten(1, (T, D)), g.t[:, T * D:]


CASES = [
    # rows, T, V, D, kind, index, extra
    (1, 1, 1, 1, "uniform", torch.int32, 0),
    (1, 47, 128, 32, "uniform", torch.int32, 0),
    (1024, 47, 128, 32, "uniform", torch.uint8, 256),
    (300, 47, 128, 32, "skewed", torch.int64, 3),
    (513, 7, 61, 33, "skewed", torch.uint8, 1),
    (65, 129, 300, 3, "uniform", torch.int32, 0),
    (400, 33, 5000, 129, "skewed", torch.int64, 1),
    (8, 512, 40000, 1031, "uniform", torch.int32, 0),
    (16, 1024, 70001, 40, "skewed", torch.int32, 8),
    (20, 1000, 3, 17, "equal", torch.int32, 0),
    (31, 1000, 900, 9, "equal", torch.int64, 0),
    (50, 10, 40, 64, "empty", torch.int32, 2),
    (3, 5, 200, 2500, "uniform", torch.int32, 0),
    (200, 1024, 1500, 8, "skewed", torch.int32, 0),     # over 131,072 tokens: the larger sorting tile
    (2, 3, 255, 5, "uniform", torch.int32, 0),
    (2, 300, 256, 16, "skewed", torch.int32, 0),        # keys 0 .. 256 need a second sorting pass
    (1200, 64, 257, 48, "skewed", torch.int32, 0),
    (77, 13, 500, 70, "uniform", torch.int64, 5),       # several blocks of rows and columns of the one-hot product
    (77, 13, 512, 2, "skewed", torch.int64, 0),
    (40, 300, 33, 31, "uniform", torch.int32, 1),
    (40, 300, 128, 1, "uniform", torch.int32, 1),
    (16, 256, 9000, 300, "skewed", torch.int32, 0),     # 4096 tokens: the most that one workgroup sorts
    (17, 241, 9000, 300, "skewed", torch.int32, 0),     # 4097
    (1, 127, 70000, 130, "equal", torch.int64, 0),      # too few tokens for partial sums
    (1, 128, 70000, 130, "equal", torch.int64, 0),
    (3, 1365, 200000, 20, "uniform", torch.int32, 7),   # three sorting passes in one workgroup
    (4, 2000, 200000, 20, "skewed", torch.int32, 0),    # and in several
    (1, 1, 100000, 64, "uniform", torch.int32, 0),
    (9, 100, 2500, 40, "skewed", torch.int32, 0),       # ten blocks of rows of the one-hot product
    (1100, 1000, 5000, 4, "equal", torch.int32, 0),     # three levels of partial sums
]


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("rows,T,V,D,kind,index,extra", CASES)
def test_matches_the_definition(rows, T, V, D, kind, index, extra, dtype):
    t = TYPES[dtype]
    tok = tokens(rows, T, V, kind, index, 3, extra=extra % 5)
    gen = torch.Generator("cuda").manual_seed(4)
    scale = 1.7
    e = gb.Embedding(rows, T, V, D, t, scale)
    table = torch.randn((V, D), generator=gen, device="cuda").to(t)
    g, out, gap = apart(rows, T, D, t, extra)
    before = gap.clone().view(torch.int16 if t == torch.bfloat16 else torch.int32)
    e.fwd(tok, table, out)
    torch.cuda.synchronize()
    g.check("out")
    assert torch.equal(gap.contiguous().view(before.dtype), before), "elements between rows were written"
    want = ref.embed_fwd(tok.long(), table, scale)
    f = ref.over(out, want, (ref.half(t) + 2 * ref.U) * want.abs())

    _, dout, _ = apart(rows, T, D, t, extra, offset=extra % 3,
                       fill=torch.randn((rows, T * D + extra), generator=gen, device="cuda").to(t))
    runs = []
    for _ in range(2):
        gd = Guarded((V, D), t)
        e.bwd(tok, dout, gd.t)
        torch.cuda.synchronize()
        gd.check("dtable")
        runs.append(gd.t)
    assert torch.equal(*runs), "the gradient differs from run to run"
    want, size, m = ref.embed_bwd(tok.long(), dout, V, scale)
    bound = (m[:, None] + 2) * ref.U * size
    b = ref.over(runs[0], want, bound + ref.half(t) * (want.abs() + bound))
    print(f"rows={rows} T={T} V={V} D={D} {kind} {dtype}: out={f:.2f} dtable={b:.2f}", flush=True)
    assert f <= 1 and b <= 1
    assert bool((runs[0][m == 0] == 0).all())


def test_no_tokens():
    for rows, T in ((0, 5), (5, 0)):
        e = gb.Embedding(rows, T, 9, 4, torch.float32)
        tok = torch.empty((rows, T), dtype=torch.int32, device="cuda")
        out = torch.empty((rows, T, 4), device="cuda")
        table = torch.full((9, 4), 3.0, device="cuda")
        e.fwd(tok, table, out)
        e.bwd(tok, out, table)
        assert bool((table == 0).all())


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("V,D", [(100, 40), (300, 33), (4000, 24)])
def test_non_finite_gradients_stay_in_their_place(V, D, dtype):
    """A NaN or an infinity of dout reaches its token's row and its column alone, and none from an empty token."""
    t = TYPES[dtype]
    gen = torch.Generator("cuda").manual_seed(10)
    rows, T = 60, 31
    tok = torch.randint(0, V, (rows, T), generator=gen, device="cuda", dtype=torch.int32)
    dout = torch.randn((rows, T, D), generator=gen, device="cuda").to(t)
    tok[7, 3] = tok[20, 1] = -1
    dout[7, 3] = float("nan")
    dout[20, 1] = float("inf")
    clean = dout.clone()
    clean[7, 3] = clean[20, 1] = 0
    tok[50, 2], tok[9, 9], tok[9, 10] = 5, 6, 6
    dout[50, 2, 4] = float("nan")
    dout[9, 9, D - 1] = float("inf")
    dout[9, 10, 1] = -float("inf")
    clean[50, 2, 4] = clean[9, 9, D - 1] = clean[9, 10, 1] = 0
    e = gb.Embedding(rows, T, V, D, t)
    dtable = torch.empty((V, D), dtype=t, device="cuda")
    e.bwd(tok, dout, dtable)
    want, size, m = ref.embed_bwd(tok.long(), clean, V, 1.0)
    assert bool(torch.isnan(dtable[5, 4])) and float(dtable[6, D - 1]) == float("inf")
    assert float(dtable[6, 1]) == -float("inf")
    for r, c in ((5, 4), (6, D - 1), (6, 1)):
        dtable[r, c] = want[r, c] = 0
    bound = (m[:, None] + 2) * ref.U * size
    assert ref.over(dtable, want, bound + ref.half(t) * (want.abs() + bound)) <= 1


def test_adjoint():
    """<embed(table), dout> = <table, gradient(dout)>, in integers, exactly."""
    gen = torch.Generator("cuda").manual_seed(9)
    for V, D in ((128, 32), (3000, 20)):
        tok = torch.randint(-3, V + 3, (90, 11), generator=gen, device="cuda", dtype=torch.int32)
        table, dout = (torch.randint(-8, 9, s, generator=gen, device="cuda").float() for s in ((V, D), (90, 11, D)))
        e = gb.Embedding(90, 11, V, D, torch.float32, 2.0)
        out, dtable = torch.empty_like(dout), torch.empty_like(table)
        e.fwd(tok, table, out)
        e.bwd(tok, dout, dtable)
        assert int((out.double() * dout).sum()) == int((table.double() * dtable).sum())


@pytest.mark.parametrize("V,D", [(128, 32), (5000, 96)])
def test_graph_replays_and_other_streams(V, D):
    gen = torch.Generator("cuda").manual_seed(6)
    rows, T = 200, 47
    tok = torch.randint(-1, V, (rows, T), generator=gen, device="cuda", dtype=torch.int32)
    table, dout = (torch.randn(s, generator=gen, device="cuda").bfloat16() for s in ((V, D), (rows, T, D)))
    e = gb.Embedding(rows, T, V, D, torch.bfloat16)
    out, dtable = torch.empty_like(dout), torch.empty_like(table)

    def step():
        e.fwd(tok, table, out)
        e.bwd(tok, dout, dtable)

    step()
    torch.cuda.synchronize()
    want = [out.clone(), dtable.clone()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    side = torch.cuda.Stream()
    for rep in range(4):
        out.fill_(float("nan"))
        dtable.fill_(float("nan"))
        torch.cuda.synchronize()
        if rep % 2:
            with torch.cuda.stream(side):
                step()
        else:
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(dtable, want[1]), rep


def test_offsets_past_32_bits():
    """dout of more than 2^31 elements, rows far apart: the last rows count."""
    rows, T, D, V = 2100, 2, 8, 16
    ld = 2 ** 20 + 1
    wide = torch.zeros((rows, ld), dtype=torch.bfloat16, device="cuda")
    out = wide[:, :T * D].unflatten(1, (T, D))
    tok = torch.arange(rows * T, device="cuda", dtype=torch.int32).reshape(rows, T) % V
    table = torch.arange(V * D, device="cuda").reshape(V, D).bfloat16()
    e = gb.Embedding(rows, T, V, D, torch.bfloat16)
    e.fwd(tok, table, out)
    assert torch.equal(out, table[tok.long()])
    dtable = torch.empty_like(table)
    out.fill_(1.0)
    e.bwd(tok, out, dtable)
    want = torch.bincount(tok.reshape(-1), minlength=V).bfloat16()[:, None].expand(V, D)
    assert torch.equal(dtable, want)
