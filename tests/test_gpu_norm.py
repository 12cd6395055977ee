"""GPU: group norm with an activation against its definition in 64 bits,
forward and backward, in both layouts and storage types.

The shapes cover the policy's layers, groups of one element, of one channel and of
all, odd channel and position counts, vectors that straddle channels, and groups
too large for one compute unit.  Bounds per element come from train_ref.
"""
import pytest
import torch

import train_ref as ref
from backward_implicit_gemm_amd import binding as gb
from parity import Guarded

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5


def setup_module():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    gb.lib()


def out_like(shape, layout, dtype, offset=0):
    """A guarded output of this layout: (guard, tensor)."""
    B, C, H, W = shape
    if layout == "nhwc":
        g = Guarded((B, H, W, C), dtype, offset=offset)
        return g, g.t.permute(0, 3, 1, 2)
    g = Guarded(shape, dtype, offset=offset)
    return g, g.t


def shifted(t, layout, offset):
    """t in this layout at an address `offset` elements past an aligned one."""
    _, v = out_like(t.shape, layout, t.dtype, offset)
    v.copy_(t)
    return v


def draw(shape, G, dtype, layout, seed, params, offset=0):
    gen = torch.Generator("cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    C = shape[1]
    x = shifted((n(*shape) * (0.5 + n(1, C, 1, 1).abs()) + n(1, C, 1, 1)).to(dtype), layout, offset)
    dy = shifted(n(*shape).to(dtype), layout, offset)
    return x, (1 + 0.3 * n(C)).to(params), (0.3 * n(C)).to(params), dy


def check(shape, G, act, layout, dtype, params=torch.float32, seed=1, offset=0, data=None, affine=True, eps=EPS):
    x, gamma, beta, dy = data or draw(shape, G, dtype, layout, seed, params, offset)
    if not affine:
        gamma = beta = None
    gn = gb.GroupNorm(shape, G, act, dtype, layout, eps, params)
    B, C = shape[:2]
    gy, y = out_like(shape, layout, dtype, offset)
    gm, gr = (Guarded((B, G), torch.float32) for _ in range(2))
    gn.fwd(x, gamma, beta, y, gm.t, gr.t)
    torch.cuda.synchronize()
    for g, name in ((gy, "y"), (gm, "mean"), (gr, "rstd")):
        g.check(name)
    wants = ref.norm_fwd(x, gamma, beta, G, act, eps)
    worst = {}
    for name, got, want, bound in zip(("y", "mean", "rstd"), (y, gm.t, gr.t), wants,
                                      ref.norm_fwd_bounds(x, gamma, beta, G, act, eps)):
        worst[name] = ref.over(got, want, bound)
    # without statistics the same output
    gy2, y2 = out_like(shape, layout, dtype, offset)
    gn.fwd(x, gamma, beta, y2)
    assert torch.equal(y2, y)

    mean, rstd = (w.float() for w in wants[1:])
    runs = []
    for _ in range(2):
        gdx, dx = out_like(shape, layout, dtype, offset)
        gdg, gdb = (Guarded((C,), params) for _ in range(2))
        gn.bwd(x, gamma, beta, dy, mean, rstd, dx, gdg.t, gdb.t)
        torch.cuda.synchronize()
        for g, name in ((gdx, "dx"), (gdg, "dgamma"), (gdb, "dbeta")):
            g.check(name)
        runs.append((dx, gdg.t, gdb.t))
    wants = ref.norm_bwd(x, gamma, beta, dy, mean, rstd, G, act)
    bounds = list(ref.norm_bwd_bounds(x, gamma, beta, dy, mean, rstd, G, act))
    for i in (1, 2):
        bounds[i] = bounds[i] + ref.half(params) * (wants[i].abs() + bounds[i])
    for name, got, again, want, bound in zip(("dx", "dgamma", "dbeta"), *runs, wants, bounds):
        assert torch.equal(got, again), f"{name} differs from run to run"
        worst[name] = ref.over(got, want, bound)
    print(f"{shape} G={G} {act} {layout} {dtype}: " + " ".join(f"{k}={v:.2f}" for k, v in worst.items()), flush=True)
    assert all(v <= 1 for v in worst.values()), worst


SHAPES = [
    ((1024, 128, 3, 4), 8, "relu"),      # conv1 of the policy
    ((1024, 128, 1, 2), 16, "silu"),     # conv2
    ((1, 1, 1, 1), 1, "none"),           # one element: its variance is 0
    ((5, 3, 1, 1), 3, "gelu"),           # groups of one element
    ((2, 7, 1, 1), 1, "silu"),           # one position, the channels of a group
    ((3, 1, 5, 1), 1, "relu"),           # one channel
    ((3, 4, 3, 5), 4, "gelu"),           # a channel a group (instance norm)
    ((2, 59, 11, 15), 1, "relu"),        # 59 channels, odd everything
    ((33, 96, 11, 15), 32, "gelu"),      # three channels a group
    ((7, 130, 5, 7), 13, "silu"),        # ten channels a group
    ((4, 34, 2, 3), 17, "none"),
    ((2, 512, 3, 3), 2, "relu"),
    ((300, 24, 2, 2), 4, "silu"),
    ((2, 64, 31, 33), 8, "silu"),
    ((3, 64, 32, 32), 1, "gelu"),        # 65,536 elements a group
    ((2, 48, 61, 67), 3, "silu"),        # 65,392 elements, odd plane
    ((1, 32, 150, 150), 2, "relu"),      # 360,000 elements a group
    ((1, 2100, 9, 11), 7, "gelu"),       # more channels than a row of threads
    ((1, 8, 1, 70001), 2, "silu"),       # one long row
    ((1, 20011, 1, 3), 1, "relu"),       # a prime number of channels
]


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("layout", ["nchw", "nhwc"])
@pytest.mark.parametrize("shape,G,act", SHAPES, ids=[f"{'x'.join(map(str, s))}-{g}-{a}" for s, g, a in SHAPES])
def test_matches_the_definition(shape, G, act, layout, dtype):
    check(shape, G, act, layout, TYPES[dtype])


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("layout", ["nchw", "nhwc"])
def test_activations_types_and_offsets(layout, act):
    check((37, 40, 3, 5), 5, act, layout, torch.bfloat16, torch.bfloat16, seed=3, offset=1)
    check((37, 40, 3, 5), 5, act, layout, torch.float32, seed=4, offset=3)
    check((9, 40, 3, 4), 10, act, layout, torch.bfloat16, seed=5, affine=False)


@pytest.mark.parametrize("layout", ["nchw", "nhwc"])
@pytest.mark.parametrize("shape,G", [((64, 128, 3, 4), 8), ((2, 16, 100, 101), 2)])
def test_a_mean_far_from_zero(shape, G, layout):
    """|mean| a thousand times the deviation: the variance must not be a difference of rounded squares."""
    x, gamma, beta, dy = draw(shape, G, torch.float32, layout, 7, torch.float32)
    x.mul_(0.1).add_(100.0)
    check(shape, G, "silu", layout, torch.float32, data=(x, gamma, beta, dy))


@pytest.mark.parametrize("layout", ["nchw", "nhwc"])
def test_constant_groups(layout):
    """A group of one value: variance 0, hat 0, y = act(beta) exactly."""
    shape, G = (6, 32, 3, 4), 4
    x, gamma, beta, dy = draw(shape, G, torch.float32, layout, 8, torch.float32)
    x.copy_(torch.arange(24.0, device="cuda").reshape(6, 4).repeat_interleave(8, 1)[:, :, None, None].expand(shape))
    gn = gb.GroupNorm(shape, G, "relu", torch.float32, layout, EPS)
    y = torch.empty_like(x)
    gn.fwd(x, gamma, beta, y)
    assert torch.equal(y, beta.clamp(min=0).reshape(1, 32, 1, 1).expand(shape))


@pytest.mark.parametrize("layout", ["nchw", "nhwc"])
def test_nan_and_infinity_stay_in_their_group(layout):
    shape, G = (8, 32, 3, 4), 4
    x, gamma, beta, dy = draw(shape, G, torch.float32, layout, 9, torch.float32)
    x[2, 3, 1, 1] = float("nan")
    x[5, 30, 0, 2] = float("inf")
    gn = gb.GroupNorm(shape, G, "relu", torch.float32, layout, EPS)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = (torch.empty((8, 4), device="cuda") for _ in range(2))
    gn.fwd(x, gamma, beta, y, mean, rstd)
    gn.bwd(x, gamma, beta, dy, mean, rstd, dx)
    bad = torch.zeros((8, 4), dtype=torch.bool, device="cuda")
    bad[2, 0] = bad[5, 3] = True
    full = bad.repeat_interleave(8, 1)[:, :, None, None].expand(shape)
    assert bool(torch.isnan(y[full]).all()) and bool(torch.isfinite(y[~full]).all())
    assert bool(torch.isnan(dx[full]).all()) and bool(torch.isfinite(dx[~full]).all())


@pytest.mark.parametrize("layout", ["nchw", "nhwc"])
def test_gradient_against_differences(layout):
    """Central differences of the 64-bit definition along random directions: the quotient is off by
    h^2/6 of the third derivative, here below 1e-6 of the directional derivative's size."""
    shape, G, act = (3, 12, 3, 5), 3, "silu"
    x, gamma, beta, dy = draw(shape, G, torch.float32, layout, 11, torch.float32)
    gn = gb.GroupNorm(shape, G, act, torch.float32, layout, EPS)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = (torch.empty((3, 3), device="cuda") for _ in range(2))
    dgamma, dbeta = (torch.empty(12, device="cuda") for _ in range(2))
    gn.fwd(x, gamma, beta, y, mean, rstd)
    gn.bwd(x, gamma, beta, dy, mean, rstd, dx, dgamma, dbeta)
    gen = torch.Generator("cuda").manual_seed(5)
    h = 1e-4
    for _ in range(5):
        vx, vg, vb = (torch.randn(t.shape, generator=gen, device="cuda", dtype=torch.float64) for t in (x, gamma, beta))
        f = lambda s: (ref.norm_fwd(x.double() + s * vx, gamma.double() + s * vg, beta.double() + s * vb, G, act, EPS)[0]  # noqa: E731
                       * dy.double()).sum()
        got = float((dx.double() * vx).sum() + (dgamma.double() * vg).sum() + (dbeta.double() * vb).sum())
        want = float((f(h) - f(-h)) / (2 * h))
        size = float((dx.double() * vx).abs().sum() + (dgamma.double() * vg).abs().sum()
                     + (dbeta.double() * vb).abs().sum())
        assert abs(got - want) <= 1e-5 * size, (got, want, size)


@pytest.mark.parametrize("layout", ["nchw", "nhwc"])
@pytest.mark.parametrize("shape,G", [((256, 128, 3, 4), 8), ((2, 32, 96, 96), 2)])
def test_graph_replays_and_other_streams(shape, G, layout):
    x, gamma, beta, dy = draw(shape, G, torch.bfloat16, layout, 13, torch.float32)
    gn = gb.GroupNorm(shape, G, "relu", torch.bfloat16, layout, EPS)
    B, C = shape[:2]
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = (torch.empty((B, G), device="cuda") for _ in range(2))
    dgamma, dbeta = (torch.empty(C, device="cuda") for _ in range(2))
    outs = (y, mean, rstd, dx, dgamma, dbeta)

    def step():
        gn.fwd(x, gamma, beta, y, mean, rstd)
        gn.bwd(x, gamma, beta, dy, mean, rstd, dx, dgamma, dbeta)

    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    side = torch.cuda.Stream()
    for rep in range(4):
        for t in outs:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        if rep % 2:
            with torch.cuda.stream(side):
                step()
        else:
            graph.replay()
        torch.cuda.synchronize()
        for got, w in zip(outs, want):
            assert torch.equal(got, w), rep


def test_more_than_2_31_elements():
    """Offsets past 32 bits: the last image of 2^31 elements and more against the same image alone."""
    C, H, W, G = 64, 32, 32, 8
    B = 2 ** 31 // (C * H * W) + 3
    gen = torch.Generator("cuda").manual_seed(17)
    x = torch.empty((B, C, H, W), dtype=torch.bfloat16, device="cuda")
    dy, y, dx = (torch.empty_like(x) for _ in range(3))
    x.fill_(0.5)
    dy.fill_(0.25)
    for t in (x, dy):
        t[-2:] = torch.randn((2, C, H, W), generator=gen, device="cuda").to(torch.bfloat16)
    gamma, beta = torch.rand(C, device="cuda"), torch.rand(C, device="cuda")
    mean, rstd = (torch.empty((B, G), device="cuda") for _ in range(2))
    gn = gb.GroupNorm(x.shape, G, "silu", torch.bfloat16)
    gn.fwd(x, gamma, beta, y, mean, rstd)
    gn.bwd(x, gamma, beta, dy, mean, rstd, dx)
    want = ref.norm_fwd(x[-2:], gamma, beta, G, "silu", EPS)[0]
    bound = ref.norm_fwd_bounds(x[-2:], gamma, beta, G, "silu", EPS)[0]
    assert ref.over(y[-2:], want, bound) <= 1
    want = ref.norm_bwd(x[-2:], gamma, beta, dy[-2:], mean[-2:], rstd[-2:], G, "silu")[0]
    bound = ref.norm_bwd_bounds(x[-2:], gamma, beta, dy[-2:], mean[-2:], rstd[-2:], G, "silu")[0]
    assert ref.over(dx[-2:], want, bound) <= 1


def instances(most=4_000_000):
    """The smallest shape of a grid that runs each kernel instance: {(instance, type, direction): (shape, G, layout)}."""
    found = {}
    for HW, W in ((1, 1), (2, 2), (3, 1), (4, 2), (5, 1), (6, 2), (7, 7), (8, 4), (12, 4), (15, 5), (16, 4), (20, 5),
                  (33, 3), (49, 7), (64, 8), (100, 10), (165, 15), (256, 16), (400, 20), (1024, 32), (2048, 32),
                  (4096, 64), (5000, 50)):
        for Cg in (1, 2, 3, 4, 5, 6, 8, 12, 16, 24, 32, 64, 128):
            for G in (1, 2, 3, 8, 32):
                for B in (1, 5, 600, 5000):
                    size = B * Cg * G * HW
                    if size > most:
                        continue
                    for layout, code in (("nchw", gb.GC_NCHW), ("nhwc", gb.GC_NHWC)):
                        d = gb.gc_norm_desc(B, Cg * G, HW // W, W, G, code, gb.GC_ACT_SILU, EPS)
                        for name, dt in (("f32", gb.GC_F32), ("bf16", gb.GC_BF16)):
                            for op in (gb.GC_OP_FWD, gb.GC_OP_BWD):
                                key = (gb.gc_group_norm_plan_name(op, d, dt).split(" ")[0], name)
                                if key not in found or size < found[key][0]:
                                    found[key] = (size, (B, Cg * G, HW // W, W), G, layout)
    return found


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("family", ["norm_split", "res_nchw", "res_nhwc", "res_small"])
def test_every_instance(family, dtype):
    cases = {v[1:] for k, v in instances().items() if k[0].startswith(family) and k[1] == dtype}
    assert len(cases) >= {"norm_split": 2, "res_nchw": 10, "res_nhwc": 20, "res_small": 5}[family]
    for i, (shape, G, layout) in enumerate(sorted(cases)):
        check(shape, G, ("silu", "relu", "gelu", "none")[i % 4], layout, TYPES[dtype], seed=20 + i)


@pytest.mark.parametrize("shape,G,layout,dtype", [
    ((8192, 128, 3, 4), 8, "nchw", "bf16"), ((8192, 128, 3, 4), 16, "nhwc", "bf16"),
    ((3, 256, 64, 67), 8, "nhwc", "f32"), ((4, 128, 128, 127), 4, "nchw", "bf16"),
    ((500, 96, 11, 15), 32, "nchw", "f32"), ((60000, 128, 1, 2), 16, "nchw", "bf16"),
    ((60000, 128, 1, 2), 16, "nhwc", "f32"),
], ids=str)
def test_outputs_past_the_cache(shape, G, layout, dtype):
    """Calls that move 64 MiB and more store their output past the cache."""
    check(shape, G, "gelu", layout, TYPES[dtype], seed=30)
