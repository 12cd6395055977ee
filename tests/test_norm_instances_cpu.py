"""The instances the GPU tests run are all that the planner picks: shapes drawn with
another seed, and by the ranges that the operators are timed over, get no other."""
import random

import norm_instances as ni
from perf import operators


def test_other_draws_find_no_other_instance():
    known = set(ni.instances())
    assert {k[0].split("<")[0] for k in known} == {f"{f}_{d}" for f in ("norm_split", "res_nchw", "res_nhwc", "res_small")
                                                   for d in ("fwd", "bwd")}
    rng = random.Random(77)
    for _ in range(40000):
        shape, G = ni.draw(rng)
        layout, dtype = rng.choice(ni.LAYOUTS)[0], rng.choice(ni.TYPES)[0]
        key = ni.instance(rng.choice(ni.OPS), shape, G, layout, dtype)
        assert key in known, (key, shape, G, layout)


def test_the_timed_ranges_find_no_other_instance():
    known = set(ni.instances())
    rng = random.Random(78)
    cases = [operators.draw(rng) for _ in range(60000)] + operators.listed()
    for c in cases:
        if not c["op"].startswith("norm"):
            continue
        shape = tuple(c[k] for k in ("batch", "channels", "height", "width"))
        key = ni.instance(ni.OPS[c["op"] == "norm_bwd"], shape, c["groups"], c["layout"],
                          {"float32": "f32", "bfloat16": "bf16"}[c["dtype"]])
        assert key in known, (key, c)
