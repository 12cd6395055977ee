"""GPU: the recurrent policy's training step and its actor, the library's operators run together,
against torch's 64-bit autograd on the CPU.

The reference rounds every tensor that the step stores between operators, and every gradient,
to the storage type, as the step does.  Errors are max|diff| / max|ref| per tensor: 1e-4
in fp32 (the repository's bound); in bf16 a path holds at most thirteen stored tensors behind
one another down and up again (conv, norm, conv, norm, features, norm, stream, norm, gates,
hidden, total, norm, logits), each off by a half step, 2^-8, where the reference rounds to the other
side: 13 * 2^-8.
"""
import pytest
import torch
import torch.nn.functional as F

from backward_implicit_gemm_amd import binding as gb
from backward_implicit_gemm_amd import encoder as enc
from backward_implicit_gemm_amd import policy as pol
from parity import f64, rel_err
from test_gpu_encoder import Stored

pytestmark = pytest.mark.gpu

BOUND = {torch.float32: 1e-4, torch.bfloat16: 13 * 2.0 ** -8}
DTYPES = pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])


def setup_module():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    gb.lib()


def reference(params, envs, length, maps, tokens, index, teacher, h0, reset):
    """Loss, logits, last state and gradients."""
    dtype = maps.dtype
    p = {k: v.detach().double().cpu().requires_grad_() for k, v in params.items()}
    kept = lambda v: Stored.apply(v, dtype)  # noqa: E731
    x, tok = maps.double().cpu(), tokens.long().cpu()
    y = F.relu(F.group_norm(kept(F.conv2d(x, p["w1"], stride=3)), enc.GROUPS[0], p["gamma1"], p["beta1"], 1e-5))
    y = F.silu(F.group_norm(kept(F.conv2d(kept(y), p["w2"])), enc.GROUPS[1], p["gamma2"], p["beta2"], 1e-5))
    features = kept(torch.cat([y.flatten(1), p["table"][tok].flatten(1)], 1))

    def norm(v, k):
        return kept(F.layer_norm(v, v.shape[-1:], p[f"gamma_{k}"], p[f"beta_{k}"], 1e-5))

    def project(v, k):
        return kept(v @ p[k][:, :, 0, 0].t())

    stream = project(norm(features, "in"), "win")
    gates = project(norm(stream, "gate"), "wgate").view(length, envs, 2 * pol.WIDTH)
    h, cut, out = h0.double().cpu(), reset.cpu().t(), []
    for t in range(length):
        a = torch.sigmoid(gates[t, :, :pol.WIDTH])
        h = a * torch.where(cut[t][:, None], 0.0, h) + (1 - a) * gates[t, :, pol.WIDTH:]
        out.append(h)
    total = kept(torch.stack(out).reshape(-1, pol.WIDTH)) + stream
    logits = project(norm(kept(total), "head"), "whead")
    share = torch.softmax(teacher.double().cpu(), 1)
    each = (share * (share.log() - torch.log_softmax(logits, 1).gather(1, index.long().cpu()))).sum(1)
    loss = each.mean()
    return each.detach(), logits.detach(), h.detach(), dict(zip(p, torch.autograd.grad(loss, list(p.values()))))


@DTYPES
def test_step_against_autograd(dtype):
    envs, length = 6, 35
    policy = pol.Policy(envs, length, dtype)
    data = pol.draw(envs, length, dtype)
    maps, tokens, index, teacher, h0, reset = data
    loss, logits, last, grads = reference({k: v.clone() for k, v in policy.params.items()}, envs, length, *data)
    got_last = torch.empty_like(h0)
    norm = policy.step(maps, tokens, index, teacher, h0, got_last, reset, rate=0.0, max_norm=1e9)[1]
    torch.cuda.synchronize()
    bound = BOUND[dtype]
    for name, a, b in (("logits", policy.core.logits, logits), ("loss", policy.loss, loss), ("last", got_last, last)):
        err = rel_err(f64(a), f64(b))
        print(f"{dtype} {name}: {err:.2e}", flush=True)
        assert err <= bound, (name, err)
    for k, g in grads.items():
        err = rel_err(f64(policy.grads[k]).reshape(g.shape), f64(g))
        print(f"{dtype} d{k}: {err:.2e}", flush=True)
        assert err <= bound, (k, err)
    want = torch.sqrt(sum(g.square().sum() for g in grads.values()))
    assert abs(float(norm) / float(want) - 1) <= bound


@DTYPES
def test_acting_is_the_rollout(dtype):
    """Steps one at a time, the state kept, give the rollout's logits: the recurrence runs over the same
    fp32 states, only its roundings differ, by far less than a step of the stored tensors."""
    envs, length = 7, 20
    policy = pol.Policy(envs, length, dtype)
    maps, tokens, index, teacher, h0, reset = pol.draw(envs, length, dtype)
    last = torch.empty_like(h0)
    policy.gradients(maps, tokens, index, teacher, h0, last, reset)
    actor = policy.actor(envs)
    actor.state.copy_(h0)
    logits = []
    for t in range(length):
        rows = slice(t * envs, (t + 1) * envs)
        logits.append(actor.act(maps[rows], tokens[rows], reset[:, t:t + 1]).clone())
    torch.cuda.synchronize()
    assert rel_err(f64(torch.cat(logits)), f64(policy.core.logits)) <= BOUND[dtype]
    assert rel_err(f64(actor.state), f64(last)) <= BOUND[dtype]


def test_gradients_in_a_graph():
    """Captured, the rollout's forward, backward and clipping replay to the eager bits, over other eager work."""
    envs, length = 8, 33
    policy, dtype = pol.Policy(envs, length, torch.bfloat16), torch.bfloat16
    maps, tokens, index, teacher, h0, reset = pol.draw(envs, length, dtype)

    def step():
        policy.gradients(maps, tokens, index, teacher, h0, None, reset)
        return policy.clip.clip(0.1)

    norm = step()
    torch.cuda.synchronize()
    want = [norm.clone(), policy.loss.clone()] + [g.clone() for g in policy.grads.values()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for rep in range(3):
        for g in list(policy.grads.values()) + [policy.loss]:
            g.fill_(float("nan"))
        other = pol.Policy(3, 5)
        data = pol.draw(3, 5)
        assert torch.isfinite(other.step(*data[:4], data[4], None, data[5])[0])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip([captured, policy.loss] + list(policy.grads.values()), want):
            assert torch.equal(a, b), rep
