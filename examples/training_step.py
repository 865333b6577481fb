"""A small language model trained with the library's operators and its optimizer: embedding, a
projection between two residual norms that keep their outputs in 8 bits, cross entropy against
the whole vocabulary, and SpectralAdamW on the three matrices.

    python examples/training_step.py [steps]

The task is synthetic: the target of a token is a fixed permutation of it, and some targets are
left out (-1), as padding would be.
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import spectral_correction_optimizer_amd as sco  # noqa: E402

EPS = 1e-5


class Model:
    """E [V, H] embedding, P [H, H] projection, W [V, H] output weights, two gains [H]."""

    def __init__(self, V=512, H=128, seed=1, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def normal(*shape, std):
            return torch.randn(*shape, generator=g, device=device) * std

        self.V, self.H, self.scale = V, H, math.sqrt(H)
        self.E, self.P, self.W = normal(V, H, std=0.02), normal(H, H, std=H ** -0.5), normal(V, H, std=0.02)
        self.gain = [torch.ones(H, device=device) for _ in range(2)]

    def matrices(self):
        return [self.E, self.P, self.W]

    def step(self, ids, targets):
        """Mean loss, the three matrices' gradients and the two gains'.  Between the passes only
        1 / rms and the 8-bit rows of each norm are kept."""
        x = sco.embed(self.E, ids, scale=self.scale)
        first = sco.rmsnorm(x, self.gain[0], eps=EPS)
        z = first.y @ self.P.t()
        second = sco.rmsnorm(z, self.gain[1], residual=x, eps=EPS)
        out = sco.xent(second.y, self.W, targets)

        dz, dgain1 = sco.rmsnorm_grad(out.dh, self.gain[1], second.rstd, second.kept)
        dP = sco.act_wgrad(dz, first.kept, gain=self.gain[0])
        dx, dgain0 = sco.rmsnorm_grad(dz @ self.P, self.gain[0], first.rstd, first.kept, dh=dz)
        dE = sco.embed_grad(dx, ids, self.V, scale=self.scale)
        return out.mean, [dE, dP, out.dW], [dgain0, dgain1]


def train(steps=60, tokens=2048, lr=0.01, anchor_every=10, seed=1):
    """Losses of `steps` steps."""
    model = Model(seed=seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    follow = torch.randperm(model.V, generator=g, device="cuda")
    opt = sco.SpectralAdamW([tuple(m.shape) for m in model.matrices()], device=torch.device("cuda", 0), lr=lr)
    losses = []
    for k in range(steps):
        ids = torch.randint(0, model.V, (tokens,), generator=g, device="cuda")
        targets = torch.where(torch.rand(tokens, generator=g, device="cuda") < 0.05, -1, follow[ids])
        loss, grads, dgains = model.step(ids, targets)
        if k % anchor_every == 0:
            opt.anchor_update(grads)
        opt.step(model.matrices(), grads)
        for gain, d in zip(model.gain, dgains):
            gain -= lr * d
        losses.append(loss)
    losses = torch.stack(losses).tolist()
    opt.close()
    return losses


if __name__ == "__main__":
    losses = train(int(sys.argv[1]) if len(sys.argv) > 1 else 60)
    for k in range(0, len(losses), max(1, len(losses) // 10)):
        print(f"step {k:4d}  loss {losses[k]:.4f}", flush=True)
    print(f"step {len(losses) - 1:4d}  loss {losses[-1]:.4f}", flush=True)
