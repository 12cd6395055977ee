"""GPU: the encoder's parameters follow their gradients, however small a step is.

Each step moves a parameter by rate times its gradient.  Kept in fp32 the sum of the
moves is off by at most half a step of fp32 for each (2^-24 of the value), whatever type the
kernels read; the parameters they read are that value rounded once.
"""
import pytest
import torch

import train_ref as ref
from backward_implicit_gemm_amd import binding as gb
from backward_implicit_gemm_amd import encoder as enc

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def setup_module():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    gb.lib()


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("rate", [1e-4, 0.1])
def test_parameters_are_the_sum_of_their_steps(rate, dtype):
    t, steps = TYPES[dtype], 40
    e, data = enc.Encoder(64, t), enc.draw(64, t)
    value = {k: v.double() for k, v in e.params.items()}
    moved = {k: torch.zeros_like(v) for k, v in value.items()}
    for _ in range(steps):
        e.step(*data, rate=rate, max_norm=1.0)
        for k, g in e.grads.items():
            value[k] -= rate * g.double()
            moved[k] += rate * g.double().abs()
    for k, v in e.params.items():
        # a step: the product and the difference are rounded in fp32
        off = steps * 2 * ref.U * (value[k].abs() + moved[k])
        worst = ref.over(v, value[k], off + ref.half(v.dtype) * (value[k].abs() + off))
        print(f"{k} {dtype} rate {rate}: {worst:.2f}", flush=True)
        assert worst <= 1, k


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_small_steps_lower_the_loss(dtype):
    e, data = enc.Encoder(64, TYPES[dtype]), enc.draw(64, TYPES[dtype])
    losses = [float(e.step(*data, rate=0.02, max_norm=1.0)[0]) for _ in range(200)]
    assert losses[-1] < 0.995 * losses[0], (losses[0], losses[-1])
