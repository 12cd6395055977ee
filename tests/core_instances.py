"""Every kernel instance that the recurrent core's planners pick, with a shape that reaches it.

The planners are asked (on the host) about shapes drawn over their range; of each instance
(template arguments, rows of a team of one wave or of several, stores in or past the cache, steps in
chunks or not) the smallest one is kept.
"""
import math
import random
import re

from backward_implicit_gemm_amd import binding as gb

MOST = 24_000_000       # values of a drawn tensor: past the cache begins at 64 MiB of a call's traffic
DTYPES = (gb.GC_F32, gb.GC_BF16)


def spread(rng, low, high):
    return max(low, min(high, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def count(rng, width):
    """Rows of this width: any number, or as many as there may be."""
    return max(1, spread(rng, 1, max(1, MOST // width)) if rng.random() < 0.4 else MOST // width)


def _number(name, key):
    found = re.search(rf"{key}=(\d+)", name)
    return int(found.group(1)) if found else None


def rows(rng):
    D = spread(rng, 1, 40000)
    shape = count(rng, D), D
    dtype, op = rng.choice(DTYPES), rng.choice((gb.GC_OP_FWD, gb.GC_OP_BWD))
    name = gb.gc_layer_norm_plan_name(op, gb.gc_layer_norm_desc(*shape, 1e-5, D, D, D, D), dtype)
    team = _number(name, "team")
    return ("rows", dtype, name.split("<")[0], _number(name, "N"), _number(name, "NV"), team and team > 64,
            _number(name, "past")), (op, dtype, *shape), shape[0] * D


def scan(rng):
    D = spread(rng, 1, 3000)
    B = spread(rng, 1, max(1, min(3000, MOST // D)))
    T = min(4000, count(rng, B * D))
    dtype, op = rng.choice(DTYPES), rng.choice((gb.GC_OP_FWD, gb.GC_OP_BWD))
    s = [gb.gc_strides(T * D, D)] * 5 + [gb.gc_strides(T, 1)]
    name = gb.gc_recurrence_plan_name(op, gb.gc_recurrence_desc(B, T, D, 1, *s), dtype)
    return ("scan", dtype, name.split("<")[0], _number(name, "N"), _number(name, "chunks") > 1,
            _number(name, "past")), (op, dtype, B, T, D), B * T * D


def distill(rng):
    V, K = spread(rng, 1, 200000), spread(rng, 1, 300)
    if rng.random() < 0.5:
        V = -(-V // 8) * 8      # the backward's stores depend on it
    shape = count(rng, V), V, K
    dtype, op = rng.choice(DTYPES), rng.choice((gb.GC_OP_FWD, gb.GC_OP_BWD, gb.GC_OP_STEP))
    name = gb.gc_distill_plan_name(op, gb.gc_distill_desc(*shape, 0, 0, 1.0, V, V, K, K), dtype)
    return ("distill", dtype, op, _number(name, "N"), _number(name, "NV"), _number(name, "team") > 64,
            _number(name, "past")), (op, dtype, *shape), shape[0] * V


def instances(seed=0, draws=60000):
    """{instance: shape}, the smallest shape found."""
    rng, found = random.Random(seed), {}
    for i in range(draws):
        for draw in (rows, scan, distill):
            key, shape, size = draw(rng)
            if key not in found or size < found[key][1]:
                found[key] = shape, size
    return {k: v[0] for k, v in found.items()}
