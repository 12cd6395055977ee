"""A recurrent policy on the observation encoder: training steps on rollouts, and acting.

    python -m backward_implicit_gemm_amd.policy [--envs 32] [--length 32] [--steps 20] [--dtype bf16]

The encoder's feature row is normed and projected to the width of a residual stream; a gated
recurrence over the rollout's steps adds to the stream; the normed stream gives the action
logits, which are distilled from a teacher's top logits.  The backward goes through all of it
and the encoder, and ends with the clipping of all gradients by their global norm and a plain
gradient step.  An ``Actor`` runs the same parameters one step at a time, its state kept
from call to call.  Everything but memory and the update runs in libgc; the projections are
convolutions of one position.
"""
import argparse

import torch

from . import binding as gb
from . import encoder as enc
from . import inputs

WIDTH, ACTIONS, TOP = 256, 300, 8      # the stream's width, the actions, and the teacher's entries a row


class Core:
    """The layers behind the encoder for `envs` environments of `length` steps each, rows time first,
    with every buffer of a forward pass.  ``params`` may be another core's."""

    def __init__(self, envs, length, features, dtype, params=None, seed=0, device="cuda"):
        rows = envs * length
        self.envs, self.length, self.rows, self.dtype = envs, length, rows, dtype
        gen = torch.Generator().manual_seed(seed)

        def weight(out, into):
            w = (2 * torch.rand((out, into, 1, 1), generator=gen) - 1) * into ** -0.5
            return w.to(device=device, dtype=dtype)

        shapes = {"win": (WIDTH, features), "wgate": (2 * WIDTH, WIDTH), "whead": (ACTIONS, WIDTH)}
        norms = {"in": features, "gate": WIDTH, "head": WIDTH}
        if params is None:
            params = {k: weight(*s) for k, s in shapes.items()}
            for k, n in norms.items():      # fp32 whatever the storage type
                params[f"gamma_{k}"], params[f"beta_{k}"] = torch.ones(n, device=device), torch.zeros(n, device=device)
        self.params = params
        self.norms = {k: gb.LayerNorm(rows, n, dtype, device=device) for k, n in norms.items()}
        self.convs = {k: gb.Conv((rows, i, 1, 1), (o, i, 1, 1), 1, 0, dtype, device) for k, (o, i) in shapes.items()}
        self.recurrence = gb.Recurrence(envs, length, WIDTH, dtype, device=device)

        def empty(*shape, of=dtype):
            return torch.empty(shape, dtype=of, device=device)

        self.empty = empty
        self.normed = {k: empty(rows, n) for k, n in norms.items()}
        self.stats = {k: [empty(rows, of=torch.float32) for _ in range(2)] for k in norms}
        self.stream, self.total, self.hidden = (empty(rows, WIDTH) for _ in range(3))
        self.gates, self.logits = empty(rows, 2 * WIDTH), empty(rows, ACTIONS)

    def sequences(self, rows):
        """Rows, time first, as (envs, length, width)."""
        return rows.unflatten(0, (self.length, self.envs)).transpose(0, 1)

    def halves(self, both):
        """Gate and value of rows that hold both."""
        return self.sequences(both[:, :WIDTH]), self.sequences(both[:, WIDTH:])

    def _norm(self, k, x, residual=None, total=None):
        p = self.params
        return self.norms[k].fwd(x, p[f"gamma_{k}"], p[f"beta_{k}"], self.normed[k], *self.stats[k], residual, total)[0]

    def _project(self, k, x, out):
        self.convs[k].fwd(x[:, :, None, None], self.params[k], out[:, :, None, None])
        return out

    def forward(self, features, h0=None, last=None, states=None, reset=None):
        """The logits of rows of features; reset is (envs, length)."""
        self._project("win", self._norm("in", features), self.stream)
        self._project("wgate", self._norm("gate", self.stream), self.gates)
        self.recurrence.fwd(*self.halves(self.gates), self.sequences(self.hidden), h0, last, states, reset)
        self._norm("head", self.hidden, self.stream, self.total)
        return self._project("whead", self.normed["head"], self.logits)


class Policy:
    """Encoder and core at one rollout size: parameters, gradients, and every buffer of a training step."""

    def __init__(self, envs, length, dtype=torch.float32, temperature=1.0, seed=0, device="cuda"):
        rows = envs * length
        self.encoder = enc.Encoder(rows, dtype, seed, device)
        self.width = self.encoder.features.shape[1]
        self.core = Core(envs, length, self.width, dtype, seed=seed + 1, device=device)
        self.dtype, self.device = dtype, device
        self.distill = gb.Distill(rows, ACTIONS, TOP, dtype, temperature, device=device)
        self.params = self.encoder.params | self.core.params
        self.grads = self.encoder.grads | {k: torch.empty_like(v) for k, v in self.core.params.items()}
        self.masters = self.encoder.masters | {k: v if v.dtype == torch.float32 else v.float()
                                               for k, v in self.core.params.items()}
        self.clip = gb.GradClip(list(self.grads.values()))
        c = self.core
        self.states = c.empty(*c.recurrence.states_shape, of=torch.float32)
        self.loss = c.empty(rows, of=torch.float32)
        self.dloss = torch.full((rows,), 1.0 / rows, device=device)      # the mean over the rows
        self.dlogits, self.dgates = c.empty(rows, ACTIONS), c.empty(rows, 2 * WIDTH)
        self.dnormed = {k: torch.empty_like(v) for k, v in c.normed.items()}
        self.dtotal = c.empty(rows, WIDTH)

    def _norm_back(self, k, x, dx, dtotal=None):
        p, g = self.core.params, self.grads
        self.core.norms[k].bwd(x, p[f"gamma_{k}"], self.dnormed[k], *self.core.stats[k], dx, g[f"gamma_{k}"],
                               g[f"beta_{k}"], dtotal)

    def _project_back(self, k, x, dout, dx):
        self.core.convs[k].bwd(x[:, :, None, None], self.core.params[k], dout[:, :, None, None], None,
                               dx[:, :, None, None], self.grads[k])

    def gradients(self, maps, tokens, index, teacher, h0=None, last=None, reset=None):
        """Fills ``loss``, a value a row, and ``grads``, of its mean."""
        c, d = self.core, self.dnormed
        c.forward(self.encoder.forward(maps, tokens), h0, last, self.states, reset)
        self.distill.step(c.logits, index, teacher, self.dloss, self.loss, self.dlogits)
        self._project_back("whead", c.normed["head"], self.dlogits, d["head"])
        self._norm_back("head", c.total, self.dtotal)
        c.recurrence.bwd(*c.halves(c.gates), self.states, c.sequences(self.dtotal), *c.halves(self.dgates), reset=reset)
        self._project_back("wgate", c.normed["gate"], self.dgates, d["gate"])
        self._norm_back("gate", c.stream, self.dtotal, self.dtotal)      # the stream's gradient past the core as well
        self._project_back("win", c.normed["in"], self.dtotal, d["in"])
        self._norm_back("in", self.encoder.features, d["in"])
        self.encoder.backward(maps, tokens, d["in"])

    def step(self, maps, tokens, index, teacher, h0=None, last=None, reset=None, rate=0.1, max_norm=1.0):
        """One training step; returns the mean loss before it and the gradients' norm before clipping."""
        self.gradients(maps, tokens, index, teacher, h0, last, reset)
        norm = self.clip.clip(max_norm)
        for k, v in self.masters.items():
            v.sub_(self.grads[k], alpha=rate)
            if v is not self.params[k]:
                self.params[k].copy_(v)
        return self.loss.mean(), norm

    def actor(self, envs):
        return Actor(self, envs)


class Actor:
    """The policy's parameters, as they are at each call, one step at a time for `envs` environments."""

    def __init__(self, policy, envs):
        self.encoder = enc.Encoder(envs, policy.dtype, device=policy.device)
        self.encoder.params = policy.encoder.params
        self.core = Core(envs, 1, policy.width, policy.dtype, policy.core.params, device=policy.device)
        self.state = torch.zeros((envs, WIDTH), device=policy.device)

    def act(self, maps, tokens, reset=None):
        """The logits of the next step, the state moved on; reset is (envs, 1), true where an episode starts."""
        return self.core.forward(self.encoder.forward(maps, tokens), self.state, self.state, None, reset)


def draw(envs, length, dtype=torch.float32, seed=1, device="cuda"):
    """Synthetic rollouts: (maps, tokens, index, teacher, h0, reset)."""
    maps, tokens, _ = enc.draw(envs * length, dtype, seed, device)
    gen = torch.Generator().manual_seed(seed + 1)
    teacher, index = (2 * torch.randn((envs * length, ACTIONS), generator=gen)).topk(TOP, 1)
    h0 = torch.randn((envs, WIDTH), generator=gen)
    reset = torch.rand((length, envs), generator=gen) < 0.05
    return maps, tokens, index.int().to(device), teacher.to(device), h0.to(device), reset.to(device).t()


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--envs", type=int, default=32)
    ap.add_argument("--length", type=int, default=32)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--dtype", choices=("f32", "bf16"), default="f32")
    a = ap.parse_args()
    dtype = inputs.torch_dtype(a.dtype)
    policy = Policy(a.envs, a.length, dtype)
    maps, tokens, index, teacher, h0, reset = draw(a.envs, a.length, dtype)
    for i in range(a.steps):
        loss, norm = policy.step(maps, tokens, index, teacher, h0, None, reset)
        print(f"step {i}: loss {float(loss):.4f}, gradient norm {float(norm):.4f}", flush=True)


if __name__ == "__main__":
    main()
