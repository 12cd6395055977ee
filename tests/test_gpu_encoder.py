"""GPU: the encoder's training step, the library's operators run together, against
the same step in torch's 64-bit autograd on the CPU.

The reference rounds every tensor that the step stores between operators, and every
gradient, to the storage type, as the step does: a relu mask depends on them.
Errors are max|diff| / max|ref| per tensor with the repository's bounds (1e-4
fp32, 1e-2 bf16; the bf16 chain rounds five tensors on the way down, each by
half a step of 2^-8, so twice that).
"""
import pytest
import torch
import torch.nn.functional as F

from backward_implicit_gemm_amd import binding as gb
from backward_implicit_gemm_amd import encoder as enc
from parity import TOL, f64, rel_err

pytestmark = pytest.mark.gpu


def setup_module():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    gb.lib()


class Stored(torch.autograd.Function):
    """A tensor stored in type t between operators: it and its gradient are rounded once."""

    @staticmethod
    def forward(ctx, x, t):
        ctx.t = t
        return x.to(t).double()

    @staticmethod
    def backward(ctx, g):
        return g.to(ctx.t).double(), None


def reference(params, maps, tokens, targets, batch):
    p = {k: v.detach().double().cpu().requires_grad_() for k, v in params.items()}
    x, tok, t = maps.double().cpu(), tokens.long().cpu(), targets.double().cpu()
    kept = lambda v: Stored.apply(v, maps.dtype)  # noqa: E731
    y = F.relu(F.group_norm(kept(F.conv2d(x, p["w1"], stride=3)), enc.GROUPS[0], p["gamma1"], p["beta1"], 1e-5))
    y = F.silu(F.group_norm(kept(F.conv2d(kept(y), p["w2"])), enc.GROUPS[1], p["gamma2"], p["beta2"], 1e-5))
    features = kept(torch.cat([y.flatten(1), p["table"][tok].flatten(1)], 1))
    loss = 0.5 * (features - t).square().sum(1).mean()
    grads = torch.autograd.grad(loss, list(p.values()))
    norm = torch.sqrt(sum(g.square().sum() for g in grads))
    return features.detach(), loss.detach(), dict(zip(p, grads)), norm


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_step_against_autograd(dtype):
    batch = 96
    tol = TOL["f32"] if dtype == torch.float32 else 2 * TOL["bf16"]
    e, data = enc.Encoder(batch, dtype), enc.draw(batch, dtype)
    before = {k: v.clone() for k, v in e.params.items()}
    features, loss, grads, norm = reference(before, *data, batch)
    got_loss, got_norm = e.step(*data, rate=0.0, max_norm=0.5)
    torch.cuda.synchronize()
    assert rel_err(f64(e.features), f64(features)) <= tol
    assert abs(float(got_loss) - float(loss)) <= tol * float(loss)
    assert abs(float(got_norm) - float(norm)) <= tol * float(norm)
    by = min(1.0, 0.5 / float(norm))
    for k, g in grads.items():
        err = rel_err(f64(e.grads[k]), f64(g) * by)
        print(f"{dtype} {k}: {err:.2e}", flush=True)
        assert err <= tol, (k, err)


def test_steps_lower_the_loss():
    e, data = enc.Encoder(64), enc.draw(64)
    losses = [float(e.step(*data, rate=1.0, max_norm=5.0)[0]) for _ in range(30)]
    assert losses[-1] < 0.9 * losses[0], losses


def test_step_in_a_graph():
    """A captured forward, backward and clipping replay to the eager bits."""
    e, data = enc.Encoder(128, torch.bfloat16), enc.draw(128, torch.bfloat16)
    maps, tokens, targets = data

    def step():
        off = e.forward(maps, tokens).float() - targets
        e.dfeatures.copy_(off / 128)
        e.backward(maps, tokens, e.dfeatures)
        return e.clip.clip(0.1)

    norm = step()
    torch.cuda.synchronize()
    want = [norm.clone()] + [g.clone() for g in e.grads.values()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for rep in range(3):
        for g in e.grads.values():
            g.fill_(float("nan"))
        eager = enc.Encoder(8).step(*enc.draw(8))      # other work between replays
        torch.cuda.synchronize()
        assert torch.isfinite(eager[0])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip([captured] + list(e.grads.values()), want):
            assert torch.equal(a, b), rep
