"""GPU: every kernel instance of group norm against the definition in 64 bits, each at
the smallest drawn shape that gets it, with stores in and past the cache."""
import pytest

import norm_instances as ni
import test_gpu_norm as norm

pytestmark = pytest.mark.gpu

setup_module = norm.setup_module
FAMILIES = [f"{f}_{d}" for f in ("norm_split", "res_nchw", "res_nhwc", "res_small") for d in ("fwd", "bwd")]


@pytest.mark.parametrize("past", [0, 1], ids=["cached", "past the cache"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("family", FAMILIES)
def test_every_instance(family, dtype, past):
    cases = {v[1:] for k, v in ni.instances().items() if k[0].startswith(family + "<") and k[1:] == (f"past={past}", dtype)}
    assert cases
    for i, (shape, G, layout, _) in enumerate(sorted(cases)):
        norm.check(shape, G, ("silu", "relu", "gelu", "none")[i % 4], layout, norm.TYPES[dtype], seed=50 + i, offset=i % 2)
