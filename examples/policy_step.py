"""A small language model adapted with the library's operators and its optimizer: layer norms, the
clipped policy loss with a KL term against a frozen copy of the model (or the preference loss of paired
answers), gradient clipping and SpectralAdamW on the three matrices.

    python examples/policy_step.py [steps] [policy | preference]

The task is synthetic: of each sequence the first tokens are a prompt, which is not trained on, and an
answer's token is good where it is a fixed permutation of the token before it.
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import spectral_correction_optimizer_amd as sco  # noqa: E402

EPS = 1e-5


class Model:
    """E [V, H] embedding, P [H, H] projection, W [V, H] output weights, two layer norms."""

    def __init__(self, V=256, H=96, seed=1, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def normal(*shape, std):
            return torch.randn(*shape, generator=g, device=device) * std

        self.V, self.H, self.scale = V, H, math.sqrt(H)
        self.E, self.P, self.W = normal(V, H, std=0.05), normal(H, H, std=H ** -0.5), normal(V, H, std=0.05)
        self.gain = [torch.ones(H, device=device) for _ in range(2)]
        self.bias = [torch.zeros(H, device=device) for _ in range(2)]

    def matrices(self):
        return [self.E, self.P, self.W]

    def vectors(self):
        return self.gain + self.bias

    def copy(self):
        """A frozen copy, the reference model."""
        other = Model.__new__(Model)
        other.__dict__.update(self.__dict__)
        other.E, other.P, other.W = (m.clone() for m in self.matrices())
        other.gain, other.bias = [v.clone() for v in self.gain], [v.clone() for v in self.bias]
        return other

    def forward(self, ids):
        """The last norm, and the first one, which is kept in 8 bits for the backward pass."""
        x = sco.embed(self.E, ids, scale=self.scale)
        first = sco.layernorm(x, self.gain[0], bias=self.bias[0], eps=EPS)
        last = sco.layernorm(first.y @ self.P.t(), self.gain[1], bias=self.bias[1], residual=x, eps=EPS, keep=False)
        return first, last

    def logp(self, ids, targets):
        return sco.token_logp(self.forward(ids)[1].y, self.W, targets)

    def step(self, ids, loss):
        """loss(last hidden states, W) is one of the library's losses with gradients; returns it, the three matrices'
        gradients, and the norms'."""
        first, last = self.forward(ids)
        out = loss(last.y, self.W)
        dz, dgain1, dbias1 = sco.layernorm_grad(out.dh, self.gain[1], last.rstd, h=last.h, mean=last.mean)
        # the projection's input is n * gain + bias, of which n is kept
        dP = sco.act_wgrad(dz, first.kept, gain=self.gain[0]) + torch.outer(dz.sum(0), self.bias[0])
        dx, dgain0, dbias0 = sco.layernorm_grad(dz @ self.P, self.gain[0], first.rstd, kept=first.kept, dh=dz)
        dE = sco.embed_grad(dx, ids, self.V, scale=self.scale)
        return out, [dE, dP, out.dW], [dgain0, dgain1, dbias0, dbias1]


class Batch:
    """Sequences of `length` tokens, the first third of each a prompt; answers sampled from a model."""

    def __init__(self, model, follow, sequences, length, g):
        T = sequences * length
        self.ids = torch.randint(0, model.V, (T,), generator=g, device=follow.device)
        logits = model.forward(self.ids)[1].y @ model.W.t()
        sampled = torch.multinomial(torch.softmax(logits, 1), 1, generator=g).squeeze(1)
        good = torch.rand(T, generator=g, device=follow.device) < 0.3  # some answers are shown
        sampled = torch.where(good, follow[self.ids], sampled)
        answer = torch.arange(T, device=follow.device) % length >= length // 3
        self.targets = torch.where(answer, sampled, torch.full_like(sampled, -1))
        reward = (sampled == follow[self.ids]).float()
        mean = reward[answer].mean()
        self.advantages = (reward - mean) / (reward[answer].std() + 1e-4)
        self.starts = torch.arange(0, T + 1, length, device=follow.device)
        # pairs of answers: the better sequence first
        score = torch.where(answer, reward, torch.zeros_like(reward)).view(sequences // 2, 2, length)
        swap = score[:, 0].sum(1) < score[:, 1].sum(1)

        def ordered(t):
            t = t.view(sequences // 2, 2, length)
            return torch.where(swap[:, None, None], t.flip(1), t).reshape(-1).contiguous()

        self.pair_ids, self.pair_targets = ordered(self.ids), ordered(self.targets)


def train(steps=20, loss="policy", sequences=64, length=24, lr=0.003, max_norm=1.0, seed=1):
    """Losses of `steps` steps, and the global norms of their gradients before clipping."""
    model = Model(seed=seed)
    reference = model.copy()
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    follow = torch.randperm(model.V, generator=g, device="cuda")
    opt = sco.SpectralAdamW([tuple(m.shape) for m in model.matrices()], device=torch.device("cuda", 0), lr=lr)
    losses, norms = [], []
    for k in range(steps):
        if k % 2 == 0:  # two steps on each batch, so that the second one's ratios are not 1
            b = Batch(model, follow, sequences, length, g)
            old = model.logp(b.ids, b.targets)
        if loss == "policy":
            ref = reference.logp(b.ids, b.targets)
            out, grads, vectors = model.step(b.ids, lambda h, W: sco.policy_loss(
                h, W, b.targets, old, b.advantages, ref_logp=ref, clip=(0.2, 0.28), kl=0.02))
            losses.append(out.total)
        else:
            ref = reference.logp(b.pair_ids, b.pair_targets)
            out, grads, vectors = model.step(b.pair_ids, lambda h, W: sco.preference_loss(
                h, W, b.pair_targets, b.starts, ref_logp=ref, beta=0.2))
            losses.append(out.mean)
        r = sco.clip_grads(grads + vectors, max_norm)
        norms.append(r.norm)
        if k % 10 == 0:
            opt.anchor_update(grads)
        opt.step(model.matrices(), grads)
        for v, d in zip(model.vectors(), vectors):
            v -= lr * d
    opt.close()
    return torch.stack(losses).tolist(), torch.stack(norms).tolist()


if __name__ == "__main__":
    kind = sys.argv[2] if len(sys.argv) > 2 else "policy"
    losses, norms = train(int(sys.argv[1]) if len(sys.argv) > 1 else 20, kind)
    for k, (x, n) in enumerate(zip(losses, norms)):
        print(f"step {k:4d}  {kind} loss {x:.4f}  gradient norm {n:.4f}", flush=True)
