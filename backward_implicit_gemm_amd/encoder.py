"""A training step of the policy's observation encoder, from the library's operators.

    python -m backward_implicit_gemm_amd.encoder [--batch 1024] [--steps 20] [--dtype bf16]

The map of an observation goes through both convolutions, each followed by a
group norm with an activation; its discrete features are embedded; both land in
one feature row.  A squared distance to given target rows stands in for the
policy's heads.  The backward ends with the clipping of all parameter gradients by
their global norm and a plain gradient step.  Convolutions, norms, embedding and
clipping run in libgc; torch provides memory, the distance and the update.
"""
import argparse

import torch

from . import binding as gb
from . import inputs

TOKENS, VOCAB, DIM = 47, 128, 32      # the discrete features, their values, and their width
GROUPS = (8, 16)                      # groups of the two norms


class Encoder:
    """The encoder at one batch size: parameters, their gradients, and every buffer of a step."""

    def __init__(self, batch, dtype=torch.float32, seed=0, device="cuda"):
        l1, l2 = inputs.LAYER1.with_batch(batch), inputs.LAYER2.with_batch(batch)
        self.batch, self.dtype = batch, dtype
        gen = torch.Generator().manual_seed(seed)

        def weight(*shape, bound):
            return ((2 * torch.rand(shape, generator=gen) - 1) * bound).to(device=device, dtype=dtype)

        # norm parameters are fp32 whatever the storage type
        self.params = {"w1": weight(*l1.w_shape, bound=l1.w_bound), "w2": weight(*l2.w_shape, bound=l2.w_bound),
                       "table": weight(VOCAB, DIM, bound=1.0)}
        for i, layer in ((1, l1), (2, l2)):
            self.params[f"gamma{i}"] = torch.ones(layer.OC, device=device)
            self.params[f"beta{i}"] = torch.zeros(layer.OC, device=device)
        self.grads = {k: torch.empty_like(v) for k, v in self.params.items()}
        # what the update moves: fp32 copies of the bf16 parameters, in which a step below half of
        # a parameter's last place would be lost
        self.masters = {k: v if v.dtype == torch.float32 else v.float() for k, v in self.params.items()}

        self.conv1 = gb.Conv(l1.x_shape, l1.w_shape, l1.stride, 0, dtype, device)
        self.conv2 = gb.Conv(l2.x_shape, l2.w_shape, l2.stride, 0, dtype, device)
        self.norm1 = gb.GroupNorm(l1.y_shape, GROUPS[0], "relu", dtype, device=device)
        self.norm2 = gb.GroupNorm(l2.y_shape, GROUPS[1], "silu", dtype, device=device)
        self.embed = gb.Embedding(batch, TOKENS, VOCAB, DIM, dtype, device=device)
        self.clip = gb.GradClip(list(self.grads.values()))

        def empty(*shape, of=dtype):
            return torch.empty(shape, dtype=of, device=device)

        self.z1, self.y1, self.dy1, self.dz1 = (empty(*l1.y_shape) for _ in range(4))
        self.z2, self.y2, self.dy2, self.dz2 = (empty(*l2.y_shape) for _ in range(4))
        self.dx = empty(*l1.x_shape)
        self.stats1 = [empty(batch, GROUPS[0], of=torch.float32) for _ in range(2)]
        self.stats2 = [empty(batch, GROUPS[1], of=torch.float32) for _ in range(2)]
        # a feature row: the convolutions' part, then the embedding
        self.width = l2.OC * l2.OH * l2.OW
        self.features, self.dfeatures = (empty(batch, self.width + TOKENS * DIM) for _ in range(2))

    def _embedded(self, rows):
        return rows[:, self.width:].unflatten(1, (TOKENS, DIM))

    def forward(self, maps, tokens):
        p = self.params
        self.conv1.fwd(maps, p["w1"], self.z1)
        self.norm1.fwd(self.z1, p["gamma1"], p["beta1"], self.y1, *self.stats1)
        self.conv2.fwd(self.y1, p["w2"], self.z2)
        self.norm2.fwd(self.z2, p["gamma2"], p["beta2"], self.y2, *self.stats2)
        self.embed.fwd(tokens, p["table"], self._embedded(self.features))
        self.features[:, :self.width] = self.y2.flatten(1)
        return self.features

    def backward(self, maps, tokens, dfeatures):
        """Fills ``grads`` from the gradient of the feature rows."""
        p, g = self.params, self.grads
        self.embed.bwd(tokens, self._embedded(dfeatures), g["table"])
        self.dy2.copy_(dfeatures[:, :self.width].unflatten(1, self.y2.shape[1:]))
        self.norm2.bwd(self.z2, p["gamma2"], p["beta2"], self.dy2, *self.stats2, self.dz2, g["gamma2"], g["beta2"])
        self.conv2.bwd(self.y1, p["w2"], self.dz2, None, self.dy1, g["w2"])
        self.norm1.bwd(self.z1, p["gamma1"], p["beta1"], self.dy1, *self.stats1, self.dz1, g["gamma1"], g["beta1"])
        self.conv1.bwd(maps, p["w1"], self.dz1, None, self.dx, g["w1"])

    def step(self, maps, tokens, targets, rate=0.1, max_norm=1.0):
        """One training step; returns the loss before it and the gradients' norm before clipping."""
        off = self.forward(maps, tokens).float() - targets
        self.dfeatures.copy_(off / self.batch)
        self.backward(maps, tokens, self.dfeatures)
        norm = self.clip.clip(max_norm)
        for k, v in self.masters.items():
            v.sub_(self.grads[k], alpha=rate)
            if v is not self.params[k]:
                self.params[k].copy_(v)
        return 0.5 * off.square().sum(1).mean(), norm


def draw(batch, dtype=torch.float32, seed=1, device="cuda"):
    """Synthetic observations and targets: (maps, tokens, targets)."""
    gen = torch.Generator().manual_seed(seed)
    maps = torch.randn(inputs.LAYER1.with_batch(batch).x_shape, generator=gen).to(dtype)
    tokens = torch.randint(0, VOCAB, (batch, TOKENS), generator=gen, dtype=torch.int32)
    l2 = inputs.LAYER2
    targets = torch.randn((batch, l2.OC * l2.OH * l2.OW + TOKENS * DIM), generator=gen)
    return maps.to(device), tokens.to(device), targets.to(device)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--batch", type=int, default=1024)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--dtype", choices=("f32", "bf16"), default="f32")
    a = ap.parse_args()
    dtype = inputs.torch_dtype(a.dtype)
    encoder, data = Encoder(a.batch, dtype), draw(a.batch, dtype)
    for i in range(a.steps):
        loss, norm = encoder.step(*data)
        print(f"step {i}: loss {float(loss):.4f}, gradient norm {float(norm):.4f}", flush=True)


if __name__ == "__main__":
    main()
