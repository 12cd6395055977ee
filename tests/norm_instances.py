"""The kernel instances the planner of group norm picks, found by asking it (host
only) about shapes drawn over its whole range: each with the smallest drawn shape
that gets it.
"""
import functools
import math
import random

from backward_implicit_gemm_amd import binding as gb

OPS = (gb.GC_OP_FWD, gb.GC_OP_BWD)
LAYOUTS = (("nchw", gb.GC_NCHW), ("nhwc", gb.GC_NHWC))
TYPES = (("f32", gb.GC_F32), ("bf16", gb.GC_BF16))


def spread(rng, low, high):
    """A whole number of [low, high], spread over its logarithm."""
    return max(low, min(high, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def instance(op, shape, G, layout, dtype):
    """The kernel and its template arguments, the type and whether the output goes past the cache."""
    B, C, H, W = shape
    name = gb.gc_group_norm_plan_name(op, gb.gc_norm_desc(B, C, H, W, G, dict(LAYOUTS)[layout], gb.GC_ACT_SILU, 1e-5),
                                      dict(TYPES)[dtype]).split(" ")
    return name[0], name[-1], dtype


def draw(rng):
    """(B, C, HW, 1) and groups: few or many channels, odd sizes and multiples of up to 16, batches that
    bring the output past the cache or stay below 4 million elements."""
    def even(v):
        m = rng.choice((1, 1, 2, 4, 8, 16))
        return max(1, v // m) * m

    while True:
        few = rng.random() < 0.5
        G, Cg = spread(rng, 1, 4 if few else 256), even(spread(rng, 1, 16 if few else 4096))
        HW = even(spread(rng, 1, 300 if rng.random() < 0.5 else 20000))
        n = G * Cg * HW
        if n <= 40_000_000:
            break
    B = 17_000_000 // n + rng.randrange(1, 4) if rng.random() < 0.5 else spread(rng, 1, max(1, 4_000_000 // n))
    return (B, G * Cg, HW, 1), G


@functools.lru_cache(maxsize=None)
def instances(draws=60000, seed=1):
    """{instance: (elements, shape, groups, layout, type)}"""
    rng, found = random.Random(seed), {}
    for _ in range(draws):
        shape, G = draw(rng)
        size = math.prod(shape)
        for layout, _ in LAYOUTS:
            for dtype, _ in TYPES:
                for op in OPS:
                    key = instance(op, shape, G, layout, dtype)
                    if key not in found or size < found[key][0]:
                        found[key] = (size, shape, G, layout, dtype)
    return found
