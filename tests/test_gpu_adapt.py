"""GPU parity of the losses of given tokens (log-probabilities, policy, preference), layer norm and the
global gradient norm against their definitions in 64 bits.  The tolerances count roundings, as in
tests/test_gpu_train.py: U is half a step of float32, HALF[dtype] of the type, relative to the value."""
import math

import pytest
import torch

from tests.gpu_harness import say
from tests.test_gpu_train import DT, F64, HALF, TINY, U, _xent_case, gen, pow2, randn, sco, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# ---- losses of given tokens --------------------------------------------------------------

class Tokens:
    """Log-probabilities of the counted tokens in 64 bits (on the CPU) with the bounds of their errors, and the
    gradients of a loss from its derivatives' bounds.  The bounds are those of cross entropy's test."""

    def __init__(self, h, W, tgt, dtype):
        self.dtype, b16 = dtype, dtype == torch.bfloat16
        h, W, tgt = h.cpu().to(F64), W.cpu().to(F64), tgt.cpu()
        (T, H), V = h.shape, W.shape[0]
        self.T, self.V, self.W = T, V, W
        self.ok = (tgt >= 0) & (tgt < V)
        self.at = tgt.clamp(0, V - 1)[:, None]
        self.h = torch.where(self.ok[:, None], h, torch.zeros((), dtype=F64))
        s, smag = self.h @ W.t(), self.h.abs() @ W.abs().t()
        es = (smag * ((H + 64) * 2 * U if b16 else ((6 * (H + 64)) * 2 + 4) * U)).amax(1, keepdim=True)
        smax = s.abs().amax(1, keepdim=True)
        lse = torch.logsumexp(s, 1, keepdim=True)
        dlse = es + (8 * smax + 4 * lse.abs() + 400 + V / 64 + 16) * U
        zero = torch.zeros((), dtype=F64)
        self.logp = torch.where(self.ok, (s.gather(1, self.at) - lse)[:, 0], zero)
        self.dlogp = torch.where(self.ok, (es + dlse + 4 * U * (smax + lse.abs()))[:, 0], zero)
        self.p = torch.exp(s - lse)
        self.rel = torch.expm1(es + dlse + (8 * smax + 16) * U)

    def gradients(self, c, dc):
        """dh, dW and their tolerances for logit gradients c (softmax - onehot), c off by at most dc."""
        b16, half = self.dtype == torch.bfloat16, HALF[self.dtype]
        c, dc = torch.where(self.ok, c, 0.0)[:, None], torch.where(self.ok, dc, 0.0)[:, None]
        unit = self.p.clone().scatter_add_(1, self.at, -torch.ones_like(c))
        eu = self.p * self.rel + (2 * half if b16 else 4 * U) * self.p
        eu.scatter_(1, self.at, (self.p * self.rel).gather(1, self.at) + (half if b16 else 2 * U) *
                    unit.abs().gather(1, self.at))
        d = c * unit
        # below the smallest normal number float32 may hold zero
        ed = ((c.abs() + dc) * eu + dc * unit.abs() + 2 * U * d.abs() + TINY) * self.ok[:, None]
        dh, dW = d @ self.W, d.t() @ self.h
        terms, da, ha, wa = 1 if b16 else 6, d.abs() + ed, self.h.abs(), self.W.abs()
        tdh = ed @ wa + (terms * (self.V + 64) + 8) * 2 * U * (da @ wa) + dh.abs() * (half + 4 * U) + TINY
        tdW = ed.t() @ ha + (terms * (self.T + 64) + 8) * 2 * U * (da.t() @ ha) + dW.abs() * (half + 4 * U) + TINY
        if b16:  # dW's product takes c h in bfloat16: one rounding of each
            tdW += half * (da.t() @ ha)
        return dh, dW, tdh, tdW


def _mask(tgt, kind, V):
    """Targets of which some are not counted, by numbers on either side of the vocabulary."""
    T = tgt.numel()
    t = torch.arange(T, device=tgt.device)
    off = {"none": t < 0, "half": t % 7 < 3, "all": t >= 0, "but last": t < T - 1, "runs": t // 50 % 2 == 0}[kind]
    return torch.where(off, torch.where(t % 2 == 0, -1, V), tgt)


CASES = [(1, 1, 1, "none"), (1, 2, 8, "none"), (2, 5, 20, "but last"), (3, 130, 64, "half"), (65, 33, 257, "none"),
         (64, 1000, 72, "half"), (130, 2500, 136, "runs"), (300, 700, 520, "runs"), (40, 5001, 64, "all"),
         (513, 257, 96, "half"), (9000, 40, 8, "runs"), (200, 600, 64, "but last")]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T,V,H,kind", CASES)
def test_token_logp(T, V, H, kind, dtype):
    say(f"case: token_logp T {T} V {V} H {H} {kind} {dtype}")
    g = gen(31)
    h, W, tgt = _xent_case(g, T, V, H, dtype)
    tgt = _mask(tgt, kind, V)
    ref = Tokens(h, W, tgt, dtype)
    got = sco().token_logp(h, W, tgt)
    within("logp", got.cpu(), ref.logp, ref.dlogp)
    assert torch.equal(got, sco().token_logp(h, W, tgt))


def _policy_inputs(g, ref, clip):
    """Old log-probabilities whose ratios keep 0.05 from the clip: there the gradient jumps."""
    d = randn(g, ref.T, std=0.3).cpu().to(F64)
    for edge in (math.log1p(-clip[0]) if clip[0] < 1 else -99.0, math.log1p(clip[1])):
        d = torch.where((d - edge).abs() < 0.05, d + 0.1, d)
    old = (ref.logp - d).float()
    adv = randn(g, ref.T).cpu()
    refl = (ref.logp + randn(g, ref.T, std=0.3).cpu()).float()
    w = torch.rand(ref.T, generator=g, device="cuda").cpu()
    w[::5] = 0.0
    return old, adv, refl, w


def _policy_ref(ref, old, adv, refl, w, clip, kl):
    """Values and bounds of the policy loss and its coefficients."""
    old, A = old.to(F64), adv.to(F64)
    lo, hi = (torch.tensor(x, dtype=torch.float32).double().item() for x in clip)
    r = torch.exp(ref.logp - old)
    high, low = (A > 0) & (r > 1 + hi), (A < 0) & (r < 1 - lo)
    stopped = (high | low) & ref.ok
    bound = torch.where(high, torch.full_like(r, 1 + hi), torch.full_like(r, 1 - lo))
    loss = -A * torch.where(stopped, bound, r)
    zero = torch.zeros((), dtype=F64)
    g, slope = torch.where(stopped, zero, A * r), torch.where(stopped, zero, (A * r).abs())
    dloss = slope * torch.expm1(ref.dlogp)
    k3 = None
    if refl is not None:
        x = refl.to(F64) - ref.logp
        k3 = torch.expm1(x) - x
        dk3 = torch.expm1(x).abs() * ref.dlogp + torch.exp(x) * ref.dlogp ** 2
        loss, dloss = loss + kl * k3, dloss + kl * dk3
        g, slope = g + kl * torch.expm1(x), slope + kl * torch.exp(x)
        k3 = (torch.where(ref.ok, k3, zero), torch.where(ref.ok, dk3, zero))
    loss = torch.where(ref.ok, loss, zero)
    count = max(1, int(ref.ok.sum()))
    share = torch.full_like(loss, 1 / count) if w is None else w.to(F64)
    share = torch.where(ref.ok, share, zero)
    dloss = dloss + U * loss.abs() + TINY
    dc = share * (slope * torch.expm1(ref.dlogp) + 3 * U * g.abs())
    return (loss, dloss, (share * loss).sum(), (share * (dloss + 2 * U * loss.abs())).sum() + U * (share * loss).sum().abs() + TINY,
            k3, stopped.sum().to(F64) / count, g * share, dc, count)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("limit", [0, 1])
@pytest.mark.parametrize("T,V,H,kind", CASES)
def test_policy_loss(T, V, H, kind, limit, dtype):
    say(f"case: policy T {T} V {V} H {H} {kind} limit {limit} {dtype}")
    g = gen(32)
    clip = (0.2, 0.28)
    h, W, tgt = _xent_case(g, T, V, H, dtype)
    tgt = _mask(tgt, kind, V)
    ref = Tokens(h, W, tgt, dtype)
    old, adv, refl, w = _policy_inputs(g, ref, clip)
    for i, (kl, use_ref, use_w) in enumerate([(0.05, True, False), (0.0, False, True)]):
        rl, wt = refl if use_ref else None, w if use_w else None
        # what is given for tokens that are not counted is not looked at
        old_in, adv_in = (torch.where(ref.ok, x, math.nan).cuda() for x in (old, adv))
        args = dict(ref_logp=rl.cuda() if use_ref else None, weights=wt.cuda() if use_w else None, clip=clip, kl=kl,
                    limit=limit)
        out = sco().policy_loss(h, W, tgt, old_in, adv_in, **args)
        loss, dloss, total, dtotal, k3, clipped, c, dc, count = _policy_ref(ref, old, adv, rl, wt, clip, kl)
        within("logp", out.logp.cpu(), ref.logp, ref.dlogp)
        within("loss", out.loss.cpu(), loss, dloss)
        within("total", out.total.cpu(), total, dtotal)
        within("clipped", out.clipped.cpu(), clipped, U * clipped)
        if use_ref:
            kl_ref = k3[0].sum() / count
            within("kl", out.kl.cpu(), kl_ref, k3[1].sum() / count + 2 * U * kl_ref + TINY)
        else:
            assert out.kl is None
        dh, dW, tdh, tdW = ref.gradients(c, dc)
        within("dh", out.dh.cpu(), dh, tdh)
        within("dW", out.dW.cpu(), dW, tdW)
        for a, b in zip(out, sco().policy_loss(h, W, tgt, old_in, adv_in, **args)):
            assert a is b is None or torch.equal(a, b)


def _starts(kind, T, pairs, g):
    """Starts of 2 pairs sequences: over all tokens, with empty ones, or with tokens before and behind."""
    n = 2 * pairs
    s = torch.randint(0, T + 1, (n + 1,), generator=g, device="cuda").sort().values
    if kind == "whole":
        s[0], s[-1] = 0, T
    elif kind == "empty":
        s[:] = torch.where(torch.arange(n + 1, device="cuda") > n // 2, T, 0)
    return s


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("limit", [0, 1])
@pytest.mark.parametrize("T,V,H,kind,pairs,cut", [(1, 3, 8, "none", 1, "whole"), (7, 50, 20, "half", 2, "whole"),
                                                  (130, 700, 136, "runs", 3, "inner"), (64, 1000, 72, "none", 5, "empty"),
                                                  (300, 130, 64, "half", 40, "whole"), (40, 300, 64, "all", 2, "whole"),
                                                  (2500, 40, 8, "runs", 1, "whole"), (65, 33, 257, "none", 0, "whole")])
def test_preference_loss(T, V, H, kind, pairs, cut, limit, dtype):
    say(f"case: preference T {T} V {V} H {H} {kind} pairs {pairs} {cut} limit {limit} {dtype}")
    g = gen(33)
    h, W, tgt = _xent_case(g, T, V, H, dtype)
    tgt = _mask(tgt, kind, V)
    starts = _starts(cut, T, pairs, g)
    ref = Tokens(h, W, tgt, dtype)
    refl = (ref.logp + randn(g, T, std=0.4).cpu()).float()
    for beta, margin, eps, average, use_ref in [(0.3, 0.0, 0.0, False, True), (2.0, 0.5, 0.125, True, False)]:
        refl_in = torch.where(ref.ok, refl, math.nan).cuda() if use_ref else None
        out = sco().preference_loss(h, W, tgt, starts, ref_logp=refl_in, beta=beta, margin=margin, smoothing=eps,
                                    average=average, limit=limit)
        b = starts.tolist()
        x = torch.where(ref.ok, ref.logp - (refl.to(F64) if use_ref else 0.0), 0.0)
        beta = torch.tensor(beta, dtype=torch.float32).double().item()
        rewards, dr = torch.zeros(pairs, 2, dtype=F64), torch.zeros(pairs, 2, dtype=F64)
        share = torch.ones(pairs, 2, dtype=F64)
        for i in range(2 * pairs):
            if average:
                share[i // 2, i % 2] = 1 / max(1, int(ref.ok[b[i]:b[i + 1]].sum()))
            rewards[i // 2, i % 2] = beta * share[i // 2, i % 2] * x[b[i]:b[i + 1]].sum()
            dr[i // 2, i % 2] = beta * share[i // 2, i % 2] * ref.dlogp[b[i]:b[i + 1]].sum()
        z, dz = rewards[:, 0] - rewards[:, 1] - margin, dr.sum(1)
        sp = torch.nn.functional.softplus
        loss = (1 - eps) * sp(-z) + eps * sp(z)
        within("rewards", out.rewards.cpu(), rewards, dr + U * rewards.abs() + TINY)
        dloss = dz + U * loss + TINY  # its slope is at most 1
        within("loss", out.loss.cpu(), loss, dloss)
        n = max(1, pairs)
        within("mean", out.mean.cpu(), loss.sum() / n, dloss.sum() / n + U * loss.sum() / n)
        within("logp", out.logp.cpu(), ref.logp, ref.dlogp)
        c, dc = torch.zeros(T, dtype=F64), torch.zeros(T, dtype=F64)
        slope = (1 - eps) * torch.sigmoid(-z) - eps * torch.sigmoid(z)
        for i in range(2 * pairs):
            k = beta / pairs * share[i // 2, i % 2]
            c[b[i]:b[i + 1]] = k * slope[i // 2] * (1 - 2 * (i % 2))
            dc[b[i]:b[i + 1]] = k * (dz[i // 2] / 4 + 2 * U * slope[i // 2].abs()) + TINY
        dh, dW, tdh, tdW = ref.gradients(c, dc)
        within("dh", out.dh.cpu(), dh, tdh)
        within("dW", out.dW.cpu(), dW, tdW)


@pytest.mark.parametrize("which", ["policy", "preference"])
def test_loss_against_differences(which):
    """The float32 gradients against differences of the 64-bit loss along a random direction."""
    g = gen(34)
    T, V, H = 60, 320, 48
    h, W, tgt = _xent_case(g, T, V, H, torch.float32)
    tgt = _mask(tgt, "half", V)
    ref = Tokens(h, W, tgt, torch.float32)
    clip, kl = (0.2, 0.28), 0.1
    old, adv, refl, _ = _policy_inputs(g, ref, clip)
    starts = torch.tensor([0, 20, 31, 44, 60], device="cuda")
    if which == "policy":
        out = sco().policy_loss(h, W, tgt, old.cuda(), adv.cuda(), ref_logp=refl.cuda(), clip=clip, kl=kl)
    else:
        out = sco().preference_loss(h, W, tgt, starts, ref_logp=refl.cuda(), beta=0.7)

    def f(a, b):
        s = a @ b.t()
        lp = torch.where(ref.ok, (s.gather(1, ref.at) - torch.logsumexp(s, 1, keepdim=True))[:, 0], 0.0)
        x = torch.where(ref.ok, refl.to(F64), 0.0) - lp
        if which == "policy":
            r, A = torch.exp(lp - old.to(F64)), adv.to(F64)
            L = -torch.minimum(r * A, r.clamp(1 - clip[0], 1 + clip[1]) * A) + kl * (torch.exp(x) - x - 1)
            return L[ref.ok].mean()
        R = torch.stack([-0.7 * x[i:j].sum() for i, j in zip(starts.tolist(), starts.tolist()[1:])]).reshape(-1, 2)
        return torch.nn.functional.softplus(R[:, 1] - R[:, 0]).mean()

    dhd, dWd = torch.randn(T, H, dtype=F64), torch.randn(V, H, dtype=F64)
    h64, W64, t = h.cpu().to(F64), W.cpu().to(F64), 1e-5
    num = (f(h64 + t * dhd, W64 + t * dWd) - f(h64 - t * dhd, W64 - t * dWd)) / (2 * t)
    a, b = out.dh.cpu().to(F64), out.dW.cpu().to(F64)
    got = (a * dhd).sum() + (b * dWd).sum()
    # float32 log-probabilities and gradients: 1e-5 of the terms is 170 roundings of each; the
    # differences' own error is of order t^2
    assert abs(got - num) <= 1e-5 * ((a * dhd).abs().sum() + (b * dWd).abs().sum()) + 1e-6 * abs(num)


@pytest.mark.parametrize("dtype", DT)
def test_token_losses_of_nothing(dtype):
    """No token, no counted token, tokens that are not counted and hold NaN."""
    m, g = sco(), gen(35)
    h, W, tgt = _xent_case(g, 70, 300, 64, dtype)
    f = randn(g, 70)
    none = torch.full_like(tgt, -1)
    s = torch.tensor([0, 30, 70], device="cuda")
    assert torch.count_nonzero(m.token_logp(h, W, none)) == 0
    out = m.policy_loss(h * math.nan, W, none, f, f, ref_logp=f, kl=0.1)
    for x in out:
        assert torch.count_nonzero(x) == 0 and not x.isnan().any()
    out = m.preference_loss(h * math.nan, W, none, s, ref_logp=f)
    assert torch.equal(out.loss, torch.full_like(out.loss, math.log(2))) and out.mean.item() == out.loss[0].item()
    for x in (out.rewards, out.logp, out.dh, out.dW):
        assert torch.count_nonzero(x) == 0 and not x.isnan().any()
    e, ei, ef = h[:0], tgt[:0], f[:0]
    assert m.token_logp(e, W, ei).shape == (0,)
    out = m.policy_loss(e, W, ei, ef, ef, ref_logp=ef, kl=0.1)
    assert out.loss.shape == (0,) and out.dh.shape == (0, 64)
    for x in (out.total, out.kl, out.clipped, out.dW):
        assert torch.count_nonzero(x) == 0
    out = m.preference_loss(e, W, ei, s * 0)
    assert out.mean.item() == pytest.approx(math.log(2), rel=2 * U) and torch.count_nonzero(out.dW) == 0
    mixed = torch.where(torch.arange(70, device="cuda") % 3 == 0, -1, tgt)
    bad = torch.where((mixed >= 0)[:, None], h, torch.full_like(h, math.nan))
    for a, b in zip(m.policy_loss(h, W, mixed, f, f), m.policy_loss(bad, W, mixed, f, f)):
        assert a is b is None or torch.equal(a, b)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("limit", [0, 1])  # (1: in pieces)
def test_policy_nonfinite_and_weightless_tokens(dtype, limit):
    """A counted token with NaN states has a NaN loss and gradient and leaves the other tokens' losses; with
    weight 0 it changes no gradient but its own row's, which is zero."""
    m, g = sco(), gen(36)
    h, W, tgt = _xent_case(g, 80, 500, 64, dtype)
    f = randn(g, 80, std=0.1)
    f[20] = -1.0
    old = m.token_logp(h, W, tgt)
    w = torch.full((80,), 1 / 80, device="cuda")
    clean = m.policy_loss(h, W, tgt, old, f, weights=w, limit=limit)
    bad = h.clone()
    bad[20, 5] = math.inf
    out = m.policy_loss(bad, W, tgt, old, f, weights=w, limit=limit)
    rest = torch.arange(80, device="cuda") != 20
    assert out.loss[20].isnan() and out.total.isnan() and torch.equal(out.loss[rest], clean.loss[rest])
    assert torch.equal(out.dh[rest], clean.dh[rest]) and out.dh[20].isnan().any()
    w[20] = 0.0
    want = m.policy_loss(h, W, tgt, old, f, weights=w, limit=limit)
    # a huge ratio of a token without weight: its loss is infinite, and reaches nothing else
    far = old.clone()
    far[20] = -3e38
    out = m.policy_loss(h, W, tgt, far, f, weights=w, limit=limit)
    assert out.loss[20].isinf()
    assert torch.equal(out.total, want.total) and torch.equal(out.dh, want.dh) and torch.equal(out.dW, want.dW)
    assert torch.count_nonzero(out.dh[20]) == 0
    # and states that are not finite, of a token without weight: its own loss alone
    for x in (math.nan, math.inf):
        bad[20, 5] = x
        out = m.policy_loss(bad, W, tgt, old, f, weights=w, limit=limit)
        assert out.loss[20].isnan() and torch.equal(out.loss[rest], want.loss[rest])
        assert torch.equal(out.total, want.total) and torch.equal(out.dh, want.dh) and torch.equal(out.dW, want.dW)


@pytest.mark.parametrize("spread", [1.0, 12.0, 60.0])
@pytest.mark.parametrize("kind", ["runs", "none"])
def test_policy_many_logits(kind, spread):
    """Enough bfloat16 logits for them to be kept relative to their rows' references (2^24): also in rows whose
    targets are far from likely, where some tiles are out of the reference's reach or all are, and in rows of
    weight 0 or that are not finite."""
    m, g = sco(), gen(39)
    T, V, H, clip = 700, 24100, 72, (0.2, 0.28)
    h, W, tgt = _xent_case(g, T, V, H, torch.bfloat16)
    h[::3] *= spread  # (a power of two or not: the reference reads what the product reads)
    tgt = _mask(tgt, kind, V)
    ref = Tokens(h, W, tgt, torch.bfloat16)
    old, adv, refl, w = _policy_inputs(g, ref, clip)
    args = dict(ref_logp=refl.cuda(), weights=w.cuda() / T, clip=clip, kl=0.05)
    w = w / T
    out = m.policy_loss(h, W, tgt, old.cuda(), adv.cuda(), **args)
    loss, dloss, total, dtotal, k3, clipped, c, dc, count = _policy_ref(ref, old, adv, refl, w, clip, 0.05)
    within("logp", out.logp.cpu(), ref.logp, ref.dlogp)
    within("loss", out.loss.cpu(), loss, dloss)
    within("total", out.total.cpu(), total, dtotal)
    dh, dW, tdh, tdW = ref.gradients(c, dc)
    within("dh", out.dh.cpu(), dh, tdh)
    within("dW", out.dW.cpu(), dW, tdW)
    for a, b in zip(out, m.policy_loss(h, W, tgt, old.cuda(), adv.cuda(), **args)):
        assert torch.equal(a, b)
    # tokens of weight 0 (every fifth) whose states are not finite
    bad = h.clone()
    bad[60, 7], bad[65, 3], bad[70] = math.nan, math.inf, -math.inf
    other = m.policy_loss(bad, W, tgt, old.cuda(), adv.cuda(), **args)
    assert torch.equal(other.dW, out.dW) and torch.equal(other.dh, out.dh) and torch.equal(other.total, out.total)
    # and one with a weight: its own row, and no other
    row = 71 if kind == "runs" else 2
    row = next(t for t in range(row, T) if ref.ok[t] and t % 5)
    bad = h.clone()
    bad[row, 7] = math.nan
    other = m.policy_loss(bad, W, tgt, old.cuda(), adv.cuda(), **args)
    rest = torch.arange(T, device="cuda") != row
    assert torch.equal(other.dh[rest], out.dh[rest]) and other.dh[row].isnan().all() and other.dW.isnan().all()


def test_policy_clip_sides():
    """On either side of the clip, with advantages of either sign and none: which tokens are stopped."""
    m, g = sco(), gen(37)
    T, V, H = 6, 50, 16
    h, W, tgt = _xent_case(g, T, V, H, torch.float32)
    lp = m.token_logp(h, W, tgt)
    ratio = torch.tensor([1.5, 1.5, 0.5, 0.5, 1.5, 1.0], device="cuda")
    A = torch.tensor([2.0, -2.0, 2.0, -2.0, 0.0, 1.0], device="cuda")
    out = m.policy_loss(h, W, tgt, lp - ratio.log(), A, clip=(0.2, 0.3))
    want = torch.tensor([-2.6, 3.0, -1.0, 1.6, 0.0, -1.0], device="cuda")
    assert (out.loss - want).abs().max() < 1e-5
    assert out.clipped.item() == pytest.approx(2 / 6, rel=2 * U)
    assert [bool(torch.count_nonzero(r)) for r in out.dh] == [False, True, True, False, False, True]


def test_preference_far_apart():
    """Rewards thousands apart: the loss is their difference or zero, never infinite."""
    m, g = sco(), gen(38)
    h, W, tgt = _xent_case(g, 40, 100, 32, torch.float32)
    s = torch.tensor([0, 10, 20, 30, 40], device="cuda")
    ref = torch.zeros(40, device="cuda")
    ref[0], ref[39] = 1e6, 2e6  # the first pair's chosen one far below, the second's rejected one
    out = m.preference_loss(h, W, tgt, s, ref_logp=ref, beta=1.0)
    assert out.loss.isfinite().all() and out.loss[1] == 0.0
    assert out.loss[0].item() == pytest.approx((out.rewards[0, 1] - out.rewards[0, 0]).item(), rel=4 * U)
    assert out.dh[:20].isfinite().all() and torch.count_nonzero(out.dh[:20]) and not torch.count_nonzero(out.dh[20:])


def test_preference_starts_outside():
    """Starts beyond the tokens are taken as their ends."""
    m, g = sco(), gen(39)
    h, W, tgt = _xent_case(g, 40, 100, 32, torch.float32)
    a = m.preference_loss(h, W, tgt, torch.tensor([0, 15, 40], device="cuda"))
    b = m.preference_loss(h, W, tgt, torch.tensor([-(1 << 40), 15, 1 << 40], device="cuda"))
    for x, y in zip(a, b):
        assert torch.equal(x, y)


# ---- layer norm ----------------------------------------------------------------------------

NORM_SIZES = [(1, 1), (3, 5), (9, 64), (130, 257), (6, 512), (5, 1000), (7, 2048), (4, 2051), (3, 4100), (2, 6144),
              (2, 8192), (2, 16384), (1, 16383), (1100, 1030), (2500, 1536), (1025, 2041)]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T,H", NORM_SIZES)
def test_layernorm(T, H, dtype):
    say(f"case: layernorm T {T} H {H} {dtype}")
    g = gen(41)
    x, r = randn(g, T, H, dtype=dtype, std=0.5), randn(g, T, H, dtype=dtype)
    gain, bias = randn(g, H, dtype=dtype), randn(g, H, dtype=dtype)
    if T > 2:
        x[0].fill_(2.0)
        r[0].fill_(1.0)  # no variance: rstd = 1 / sqrt(eps), n = 0
        r[1] = r[1] * 1e-3 + 100.0  # far from 0
    eps = 2.0 ** -17  # exact in float32
    for res, b in ((r, bias), (None, None)):
        out = sco().layernorm(x, gain, bias=b, residual=res, eps=eps)
        h = x.to(F64) + (0 if res is None else res.to(F64))
        within("h", out.h, h, h.abs() * HALF[dtype])
        mean = h.mean(1)
        tiny = 1e-13 * h.abs().amax(1)  # sums of 64 bits
        within("mean", out.mean, mean, U * mean.abs() + tiny)
        rstd = 1 / ((h - mean[:, None]).square().mean(1) + eps).sqrt()
        within("rstd", out.rstd, rstd, 1.01 * U * rstd)
        n = (h - mean[:, None]) * rstd[:, None]
        dn = (tiny * rstd)[:, None] + 1e-13 * n.abs()
        y = n * gain.to(F64) + (0 if b is None else b.to(F64))
        # n as float32, the product and sum once, the store; below the normal numbers a store may be zero
        ty = y.abs() * (HALF[dtype] + 1.01 * U) + (n * gain.to(F64)).abs() * 1.01 * U + dn * gain.to(F64).abs()
        within("y", out.y, y, ty + TINY)
        nb = -(-H // 32)
        e = out.kept.e.to(torch.int32) - 127
        p = torch.zeros(T, nb * 32, dtype=F64, device="cuda")
        p[:, :H] = n
        amax, slack = p.reshape(T, nb, 32).abs().amax(2), dn.amax(1)[:, None]
        assert ((pow2(e) <= amax + slack) | (e == -120)).all()
        assert (pow2(e + 1) > amax - slack).all()
        step = pow2(e - 6).repeat_interleave(32, 1)[:, :H]
        clip = out.kept.q.abs() == 127
        within("kept", sco().act_unpack(out.kept, torch.float32), n, torch.where(clip, 1.0, 0.5) * step + dn)
    two = sco().layernorm(x, gain, eps=eps, keep=False)
    assert two.kept is None and two.h is x and torch.equal(two.y, out.y)


@pytest.mark.parametrize("dtype", DT)
def test_layernorm_rows_stay_apart(dtype):
    g = gen(42)
    x, gain = randn(g, 9, 100, dtype=dtype), randn(g, 100, dtype=dtype)
    x[1, 3], x[4, 99] = math.nan, math.inf
    out = sco().layernorm(x, gain)
    kept = sco().act_unpack(out.kept, torch.float32)
    for t in range(9):
        assert bool(out.y[t].isfinite().all()) == (t not in (1, 4))
        assert bool(kept[t].isfinite().all()) == (t not in (1, 4))
    for x in sco().layernorm(x[:0], gain)[:4]:
        assert x.shape[0] == 0


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("kept", [True, False])
@pytest.mark.parametrize("T,H", [(0, 40)] + NORM_SIZES + [(5000, 96), (2300, 1100)])
def test_layernorm_grad(T, H, kept, dtype):
    say(f"case: layernorm_grad T {T} H {H} kept {kept} {dtype}")
    g = gen(43)
    dy, dh = randn(g, T, H, dtype=dtype), randn(g, T, H, dtype=dtype)
    gain = randn(g, H, dtype=dtype)
    rstd = torch.rand(T, generator=g, device="cuda") + 0.5
    rs = rstd.to(F64)[:, None]
    if kept:
        rows = dict(kept=sco().act_pack(randn(g, T, H)))
        n = sco().act_unpack(rows["kept"], torch.float32).to(F64)
        en = torch.zeros_like(n)
    else:
        rows = dict(h=randn(g, T, H, dtype=dtype), mean=randn(g, T))
        n = (rows["h"].to(F64) - rows["mean"].to(F64)[:, None]) * rs
        en = 2.01 * U * n.abs()
    dx, dgain, dbias = sco().layernorm_grad(dy, gain, rstd, dh=dh, **rows)
    a = dy.to(F64) * gain.to(F64)
    c0, c1 = a.mean(1, keepdim=True) if H else a, (a * n).sum(1, keepdim=True) / H
    # a row's sums and their products
    terms = (64 + 8 + 3) * U
    dc0 = terms * a.abs().sum(1, keepdim=True) / H
    dc1 = (terms * (a * n).abs() + a.abs() * en).sum(1, keepdim=True) / H
    part = rs * (a.abs() + c0.abs() + n.abs() * c1.abs())
    more = rs * (dc0 + n.abs() * dc1 + en * c1.abs())
    ref = dh.to(F64) + rs * (a - c0 - n * c1)
    within("dx", dx, ref, ref.abs() * HALF[dtype] + 5 * U * (part + dh.to(F64).abs()) + more)
    dg, db = (dy.to(F64) * n).sum(0), dy.to(F64).sum(0)
    within("dgain", dgain, dg, ((T + 40) * U * (dy.to(F64) * n).abs() + dy.to(F64).abs() * en).sum(0))
    within("dbias", dbias, db, (T + 40) * U * dy.to(F64).abs().sum(0))
    dx0, dgain0, dbias0 = sco().layernorm_grad(dy, gain, rstd, **rows)
    ref = rs * (a - c0 - n * c1)
    within("dx alone", dx0, ref, ref.abs() * HALF[dtype] + 5 * U * part + more)
    assert torch.equal(dgain, dgain0) and torch.equal(dbias, dbias0)


def test_layernorm_grad_against_differences():
    """The gradient of <y, dy> + <h, dh> with respect to x, gain and bias, by differences in 64 bits."""
    g = gen(44)
    T, H, eps = 6, 72, 2.0 ** -17
    x, gain, bias = randn(g, T, H), randn(g, H), randn(g, H)
    dy, dh = randn(g, T, H), randn(g, T, H)
    out = sco().layernorm(x, gain, bias=bias, eps=eps)
    dx, dgain, dbias = sco().layernorm_grad(dy, gain, out.rstd, h=out.h, mean=out.mean, dh=dh)

    def f(z, gn, b):
        n = (z - z.mean(1, keepdim=True)) / (z.var(1, unbiased=False, keepdim=True) + eps).sqrt()
        return ((n * gn + b) * dy.double()).sum() + (z * dh.double()).sum()

    d = [torch.randn(*s, generator=g, device="cuda", dtype=F64) for s in ((T, H), (H,), (H,))]
    p, t = [v.double() for v in (x, gain, bias)], 1e-5
    num = (f(*(a + t * b for a, b in zip(p, d))) - f(*(a - t * b for a, b in zip(p, d)))) / (2 * t)
    got = [(a.double() * b) for a, b in zip((dx, dgain, dbias), d)]
    # float32: at most 100 roundings of each term and of what cancels in it; differences of order t^2
    assert abs(sum(v.sum() for v in got) - num) <= 400 * U * sum(v.abs().sum() for v in got) + 1e-6 * abs(num)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T,H", [(40, 1000), (700, 4100), (300, 2049), (9, 8191), (5, 9001), (64, 7), (33, 2048), (3000, 1501),
                                 (2100, 2047), (50, 1030)])
def test_layernorm_in_place(T, H, dtype):
    """The C entries allow h = x, h = residual, dx = dy and dx = dh."""
    say(f"case: layernorm in place T {T} H {H} {dtype}")
    m, g = sco(), gen(45)
    lib, dt, st = m.load_library(), m._DT[dtype], torch.cuda.current_stream().cuda_stream
    x, r, dy, dh = (randn(g, T, H, dtype=dtype) for _ in range(4))
    gain, bias = randn(g, H, dtype=dtype), randn(g, H, dtype=dtype)
    want = m.layernorm(x, gain, bias=bias, residual=r)
    for i in range(2):
        a = [x.clone(), r.clone()]
        y, mean, rstd = torch.empty_like(x), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        assert lib.sc_layernorm(dt, a[0].data_ptr(), a[1].data_ptr(), gain.data_ptr(), bias.data_ptr(), 1e-5, T, H,
                                a[i].data_ptr(), y.data_ptr(), mean.data_ptr(), rstd.data_ptr(), None, None, st) == 0
        assert torch.equal(a[i], want.h) and torch.equal(y, want.y)
        assert torch.equal(mean, want.mean) and torch.equal(rstd, want.rstd)
    n = m._workspace_bytes("sc_layernorm_grad_workspace", T, H)
    for kept in (True, False):
        rows = dict(kept=want.kept) if kept else dict(h=want.h, mean=want.mean)
        dx, dgain, dbias = m.layernorm_grad(dy, gain, want.rstd, dh=dh, **rows)
        src = [want.kept.q.data_ptr(), want.kept.e.data_ptr(), None, None] if kept else \
            [None, None, want.h.data_ptr(), want.mean.data_ptr()]
        for i in range(2):
            a = [dy.clone(), dh.clone()]
            dg, db, ws = (torch.empty(k, device="cuda") for k in (H, H, n // 4))
            assert lib.sc_layernorm_grad(dt, a[0].data_ptr(), gain.data_ptr(), want.rstd.data_ptr(), *src,
                                         a[1].data_ptr(), T, H, a[i].data_ptr(), dg.data_ptr(), db.data_ptr(),
                                         ws.data_ptr(), n, st) == 0
            assert torch.equal(a[i], dx) and torch.equal(dg, dgain) and torch.equal(db, dbias)


# ---- global gradient norm ------------------------------------------------------------------

def _grads(g, sizes, dtypes, std=1.0):
    """Tensors inside one buffer of each type, a sentinel of 7 between them; the buffers."""
    out, bufs = [], {}
    for dt in set(dtypes):
        bufs[dt] = torch.full((sum(sizes) + 3 * len(sizes) + 3,), 7.0, dtype=dt, device="cuda")
    at = dict.fromkeys(bufs, 1)
    for n, dt in zip(sizes, dtypes):
        v = bufs[dt][at[dt]:at[dt] + n]
        v.copy_(randn(g, n, dtype=dt, std=std))
        at[dt] += n + 3
        out.append(v)
    return out, bufs


SIZES = [[1], [0, 5, 0], [8191, 8192, 8193], [7, 1, 3000, 64, 9, 100001], [int(3 + (i * 7919) % 900) for i in range(300)],
         [3000017, 12]]


@pytest.mark.parametrize("mixed", [False, True])
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
def test_clip_grads(sizes, dtype, mixed):
    say(f"case: clip {len(sizes)} tensors, largest {max(sizes)} {dtype} mixed {mixed}")
    m, g = sco(), gen(51)
    dts = [DT[i % 2] if mixed else dtype for i in range(len(sizes))]
    grads, bufs = _grads(g, sizes, dts)
    total = sum((v.to(F64) ** 2).sum() for v in grads)
    within("sumsq", m.grad_sumsq(grads), total, 1e-12 * total)
    for limit in (0.37 * float(total.sqrt()), 2 * float(total.sqrt()) + 1, 0.0, math.inf):
        f32 = torch.tensor(limit, dtype=torch.float32).double().item()
        before = {dt: b.clone() for dt, b in bufs.items()}
        outs, obufs = _grads(g, sizes, dts)
        marks = {dt: b.clone() for dt, b in obufs.items()}
        r = m.clip_grads(grads, limit, out=outs)
        within("norm", r.norm, total.sqrt(), U * 1.01 * total.sqrt())
        scale = (f32 / (total.sqrt() + 1e-6)).clamp(max=1.0)
        within("scale", r.scale, scale, U * 1.01 * scale)
        for v, o in zip(grads, outs):
            assert torch.equal(o, (v.float() * r.scale).to(v.dtype))  # one rounding of the float32 product
        for dt, b in bufs.items():
            assert torch.equal(b, before[dt])
        # nothing between the outputs was written
        for v, o in zip(grads, outs):
            o.copy_(torch.zeros_like(o))
        probe, pbufs = _grads(gen(51), sizes, dts)
        for v in probe:
            v.zero_()
        for dt in obufs:
            assert torch.equal((obufs[dt] == 7.0) | (obufs[dt] == 0.0), torch.ones_like(obufs[dt], dtype=torch.bool))
            assert torch.equal(obufs[dt] == 7.0, pbufs[dt] == 7.0) and marks[dt].shape == obufs[dt].shape
    want = [(v.float() * m.clip_grads(grads, 0.25, out=[torch.empty_like(v) for v in grads]).scale).to(v.dtype) for v in grads]
    r = m.clip_grads(grads, 0.25)  # in place
    for v, w, t in zip(grads, want, r.grads):
        assert torch.equal(v, w) and t is v


def test_clip_known_sum_and_shapes():
    """The sum of squares of two shards, and tensors of more than one axis."""
    m, g = sco(), gen(52)
    a, b = randn(g, 33, 70), randn(g, 5, 3, 11)
    s = m.grad_sumsq([a]) + m.grad_sumsq([b])
    whole = m.clip_grads([a, b], 1.0, out=[torch.empty_like(a), torch.empty_like(b)])
    first = m.clip_grads([a], 1.0, out=[torch.empty_like(a)], sumsq=s)
    assert abs(first.norm.item() - whole.norm.item()) <= 2 * U * whole.norm.item()
    within("shard", first.grads[0], whole.grads[0].to(F64), 4 * U * whole.grads[0].abs().to(F64) + TINY)


def test_clip_extremes():
    """Squares out of float32's range, and values that are not finite."""
    m = sco()
    big = torch.full((1000,), 3e38, device="cuda")
    r = m.clip_grads([big], 1.0)
    # the norm itself is above float32's largest number
    assert r.norm.isinf() and r.scale.item() == pytest.approx(1 / (3e38 * math.sqrt(1000)), rel=1e-2)
    small = torch.full((1000,), 1e-30, device="cuda")
    s = m.grad_sumsq([small]).item()
    assert s == pytest.approx(1000 * float(torch.tensor(1e-30)) ** 2, rel=1e-12)
    x = torch.ones(100, device="cuda")
    x[3] = math.inf
    r = m.clip_grads([x], 1.0)
    assert r.norm.isinf() and r.scale.item() == 0.0 and x[3].isnan() and torch.count_nonzero(x) == 1
    x = torch.ones(100, device="cuda")
    x[99] = math.nan
    r = m.clip_grads([x], 1.0)
    assert r.norm.isnan() and r.scale.isnan() and x.isnan().all()
    e = torch.empty(0, device="cuda")
    r = m.clip_grads([e], 1.0)
    assert r.norm.item() == 0.0 and r.scale.item() == 1.0


def test_clip_beyond_32_bits():
    """A tensor of more than 2^32 bytes and 2^31 elements."""
    m = sco()
    n = (1 << 31) + 13
    x = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    x[0], x[-1], x[1 << 30] = 3.0, 4.0, 12.0
    r = m.clip_grads([x], 1.0)
    assert r.norm.item() == 13.0
    assert [x[i].item() for i in (0, -1, 1 << 30)] == [(torch.tensor(v) * r.scale.cpu()).bfloat16().item() for v in (3.0, 4.0, 12.0)]
    assert torch.count_nonzero(x).item() == 3


# ---- streams and graphs ----------------------------------------------------------------------

def test_adapt_other_stream_and_graph_replays():
    """The operators on a stream of their own, and captured into a graph that is replayed on new
    inputs, with eager calls between, give the eager results bit for bit."""
    m, g = sco(), gen(61)
    V, H, T = 600, 128, 200
    W, gain, bias = randn(g, V, H, dtype=torch.bfloat16, std=0.3), randn(g, H, dtype=torch.bfloat16), randn(g, H, dtype=torch.bfloat16)
    x = randn(g, T, H, dtype=torch.bfloat16)
    tgt = torch.randint(-1, V, (T,), generator=g, device="cuda")
    adv, ref = randn(g, T), randn(g, T) - 6
    starts = torch.tensor([0, 40, 90, 170, 200], device="cuda")

    def step():
        n = m.layernorm(x, gain, bias=bias, residual=x)
        lp = m.token_logp(n.y, W, tgt)
        a = m.policy_loss(n.y, W, tgt, lp + 0.1 * adv, adv, ref_logp=ref, kl=0.1)
        b = m.preference_loss(n.y, W, tgt, starts, ref_logp=ref)
        dx, dgain, dbias = m.layernorm_grad(a.dh, gain, n.rstd, kept=n.kept, dh=b.dh)
        dx2, _, _ = m.layernorm_grad(a.dh, gain, n.rstd, h=n.h, mean=n.mean, dh=b.dh)
        grads = [a.dW, dgain, dbias]
        r = m.clip_grads(grads, 0.5, out=[torch.empty_like(v) for v in grads])
        return [n.h, n.y, n.mean, n.rstd, lp, *a, *b, dx, dgain, dbias, dx2, r.norm, r.scale, *r.grads]

    eager = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(eager, got):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(4):
        x.copy_(randn(g, T, H, dtype=torch.bfloat16))
        # counted tokens: some, others, none, all
        tgt.copy_(torch.randint(-1 if k < 2 else 0, V, (T,), generator=g, device="cuda"))
        if k == 2:
            tgt.fill_(-1)
        want = [t.clone() for t in step()]
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, out):
            assert torch.equal(a, b), k


# more output tiles than workgroups run at once, rows of tokens that are left out in whole tiles
@pytest.mark.parametrize("dtype", DT)
def test_policy_many_tiles(dtype):
    T, V, H = 700, 70003, 72
    say(f"case: policy many tiles T {T} V {V} H {H} {dtype}")
    g = gen(62)
    h, W, tgt = _xent_case(g, T, V, H, dtype)
    tgt[:400] = -1
    ref = Tokens(h, W, tgt, dtype)
    old, adv, refl, _ = _policy_inputs(g, ref, (0.2, 0.2))
    out = sco().policy_loss(h, W, tgt, old.cuda(), adv.cuda(), ref_logp=refl.cuda(), kl=0.02)
    loss, dloss, _, _, _, _, c, dc, _ = _policy_ref(ref, old, adv, refl, None, (0.2, 0.2), 0.02)
    within("loss", out.loss.cpu(), loss, dloss)
    dh, dW, tdh, tdW = ref.gradients(c, dc)
    within("dh", out.dh.cpu(), dh, tdh)
    within("dW", out.dW.cpu(), dW, tdW)


# whole tiles of every shape and several rounds of them, with the last round cut along k: rows and columns that end
# inside a tile, more tokens left out than a tile has
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T,V,H,masked", [(1500, 5000, 1032, 700), (900, 16000, 520, 100), (700, 40000, 257, 400)])
def test_policy_large_tiles(T, V, H, masked, dtype):
    say(f"case: policy large tiles T {T} V {V} H {H} masked {masked} {dtype}")
    g = gen(63)
    h, W, tgt = _xent_case(g, T, V, H, dtype)
    tgt[torch.randperm(T, generator=g, device="cuda")[:masked]] = -1
    ref = Tokens(h, W, tgt, dtype)
    old, adv, refl, _ = _policy_inputs(g, ref, (0.2, 0.2))
    args = (h, W, tgt, old.cuda(), adv.cuda())
    out = sco().policy_loss(*args, ref_logp=refl.cuda(), kl=0.02)
    loss, dloss, _, _, _, _, c, dc, _ = _policy_ref(ref, old, adv, refl, None, (0.2, 0.2), 0.02)
    within("loss", out.loss.cpu(), loss, dloss)
    dh, dW, tdh, tdW = ref.gradients(c, dc)
    within("dh", out.dh.cpu(), dh, tdh)
    within("dW", out.dW.cpu(), dW, tdW)
    # and nearer in the mean: each element of the gradients has a few roundings of its own
    for got, want in ((out.dh, dh), (out.dW, dW)):
        off = (got.cpu().to(F64) - want).norm() / want.norm()
        assert off <= (4 * HALF[dtype] if dtype == torch.bfloat16 else 2.0 ** -16), off
    for _ in range(3):
        for a, b in zip(out, sco().policy_loss(*args, ref_logp=refl.cuda(), kl=0.02)):
            assert torch.equal(a, b)


# few tokens: the weights' gradient goes down the vocabulary with all tokens in registers; columns and rows that end
# inside a panel or a step, more panels than one, tokens of one and of two tiles, pieces
@pytest.mark.parametrize("limit", [0, 1])
@pytest.mark.parametrize("T,V,H,kind", [(1, 3000, 300, "none"), (64, 5000, 520, "half"), (65, 4099, 1025, "none"),
                                        (96, 20000, 264, "runs"), (128, 70001, 72, "half"), (128, 200, 2048, "none"),
                                        (100, 6400, 64, "all"), (128, 1000, 8191, "half")])
def test_policy_few_tokens(T, V, H, kind, limit):
    say(f"case: policy few tokens T {T} V {V} H {H} {kind} limit {limit}")
    g = gen(64)
    h, W, tgt = _xent_case(g, T, V, H, torch.bfloat16)
    tgt = _mask(tgt, kind, V)
    ref = Tokens(h, W, tgt, torch.bfloat16)
    old, adv, refl, _ = _policy_inputs(g, ref, (0.2, 0.2))
    args = (h, W, tgt, old.cuda(), adv.cuda())
    out = sco().policy_loss(*args, ref_logp=refl.cuda(), kl=0.02, limit=limit)
    _, _, _, _, _, _, c, dc, _ = _policy_ref(ref, old, adv, refl, None, (0.2, 0.2), 0.02)
    dh, dW, tdh, tdW = ref.gradients(c, dc)
    within("dh", out.dh.cpu(), dh, tdh)
    within("dW", out.dW.cpu(), dW, tdW)
    for _ in range(2):
        for a, b in zip(out, sco().policy_loss(*args, ref_logp=refl.cuda(), kl=0.02, limit=limit)):
            assert torch.equal(a, b)


# few tokens against many columns: the logits' tiles that are made for reading the weights
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T,V,H,kind", [(64, 20000, 520, "half"), (5, 16384, 1000, "none"), (128, 17001, 136, "none"),
                                        (100, 40000, 2048, "runs"), (65, 33000, 77, "but last")])
def test_token_logp_few_tokens(T, V, H, kind, dtype):
    say(f"case: token_logp few tokens T {T} V {V} H {H} {kind} {dtype}")
    g = gen(65)
    h, W, tgt = _xent_case(g, T, V, H, dtype)
    tgt = _mask(tgt, kind, V)
    ref = Tokens(h, W, tgt, dtype)
    got = sco().token_logp(h, W, tgt)
    within("logp", got.cpu(), ref.logp, ref.dlogp)
    for limit in (0, 1):
        out = sco().policy_loss(h, W, tgt, got, torch.ones_like(got), limit=limit)
        within("logp of the loss", out.logp.cpu(), ref.logp, ref.dlogp)
        c = torch.where(ref.ok, 1.0, 0.0).to(F64) / max(1, int(ref.ok.sum()))  # every ratio is 1, next to none
        dh, dW, tdh, tdW = ref.gradients(c, c * (torch.expm1(2 * ref.dlogp) + 4 * U))
        within("dh", out.dh.cpu(), dh, tdh)
        within("dW", out.dW.cpu(), dW, tdW)


# ---- the operators together ------------------------------------------------------------------

@pytest.mark.parametrize("loss", ["policy", "preference"])
def test_example_runs(loss):
    """The example's model, adapted by its own loop."""
    from examples.policy_step import train
    losses, norms = train(steps=6, loss=loss)
    assert len(losses) == len(norms) == 6
    assert all(math.isfinite(x) for x in losses) and all(0 < x < math.inf for x in norms)
    if loss == "preference":  # model and reference are the same: nothing is preferred yet
        assert losses[0] == pytest.approx(math.log(2), rel=1e-5)


@pytest.mark.parametrize("loss", ["policy", "preference"])
def test_example_gradients_against_differences(loss):
    """The loss changes along the gradients by their squared norm, to first order.  The first norm's checkpoint (half
    a step of 1/64 of a block's largest power of two, at most 1% of the largest value, twice) bounds what
    the gradients that read it are off by; float32 losses are off by 80 U."""
    from examples.policy_step import Batch, Model
    g = gen(71)
    m = Model(V=64, H=64, seed=3)
    ref_model = Model(V=64, H=64, seed=4)
    follow = torch.randperm(64, generator=g, device="cuda")
    b = Batch(m, follow, 16, 18, g)
    old = m.logp(b.ids, b.targets) + 0.05  # no ratio near the clip
    ref = ref_model.logp(b.ids, b.targets)
    pair_ref = ref_model.logp(b.pair_ids, b.pair_targets)
    if loss == "policy":
        f = lambda h, W: sco().policy_loss(h, W, b.targets, old, b.advantages, ref_logp=ref, kl=0.1)
        run = lambda: m.step(b.ids, f)
    else:
        f = lambda h, W: sco().preference_loss(h, W, b.pair_targets, b.starts, ref_logp=pair_ref, beta=0.5)
        run = lambda: m.step(b.pair_ids, f)
    value = lambda out: float(out.total if loss == "policy" else out.mean)
    out, grads, vectors = run()
    params, every = m.matrices() + m.vectors(), grads + vectors
    norm2 = sum((d.double() ** 2).sum() for d in every)
    t = 1e-3 / float(norm2.sqrt())
    found = []
    for sign in (1, -1):
        for p, d in zip(params, every):
            p.add_(sign * t * d)
        found.append(value(run()[0]))
        for p, d in zip(params, every):
            p.sub_(sign * t * d)
    slope = (found[0] - found[1]) / (2 * t)
    # the losses' terms, of which 80 U each is float32's: of order 1 and, for a policy, as large as the advantages
    size = 1 + float(b.advantages.abs().max())
    assert abs(slope - float(norm2)) <= 80 * U * size / t + 0.04 * float(norm2)


def test_optimizer_step_clips():
    """SpectralAdamW.step with max_norm is clip_grads in place, then the step."""
    m, g = sco(), gen(72)
    shapes = [(96, 64), (64, 160)]
    runs = []
    for way in range(2):
        opt = m.SpectralAdamW(shapes, device=torch.device("cuda", 0))
        gg = gen(73)
        W, G = [randn(gg, *s) for s in shapes], [randn(gg, *s) for s in shapes]
        opt.anchor_update([x.clone() for x in G])
        if way == 0:
            r = opt.step(W, G, max_norm=0.5)
        else:
            r = m.clip_grads(G, 0.5)
            assert opt.step(W, G) is None
        torch.cuda.synchronize()
        runs.append([*W, *G, r.norm, r.scale])
        opt.close()
    for a, b in zip(*runs):
        assert torch.equal(a, b)
    total = sum((x.to(F64) ** 2).sum() for x in runs[0][2:4]).sqrt()
    assert abs(total.item() - 0.5) < 1e-5


def test_clip_refuses_other_lists():
    m = sco()
    x, y = torch.ones(4, 6, device="cuda"), torch.ones(6, 4, device="cuda")
    for bad in ([x.t()], [x.half()], [x.cpu()], [x, y.cpu()], [x, 3], [x, x.t()]):
        with pytest.raises(ValueError):
            m.clip_grads(bad, 1.0)
    for out in ([], [y], [x.bfloat16()], [torch.ones(6, 4, device="cuda").t()]):
        with pytest.raises(ValueError):
            m.clip_grads([x], 1.0, out=out)
    for s in (torch.ones((), device="cuda"), torch.ones(1, dtype=F64, device="cuda"), torch.ones((), dtype=F64)):
        with pytest.raises(ValueError):
            m.clip_grads([x], 1.0, sumsq=s)
    with pytest.raises(m.ScoptError):
        m.clip_grads([x], -1.0)
    # a tensor twice, tensors that overlap, outputs that are other inputs' memory
    b = torch.ones(100, device="cuda")
    for grads, out in (([x, x], None), ([b[:60], b[50:]], None), ([b[:50], b[50:]], [b[50:], b[:50]]),
                       ([b[:40]], [b[1:41]]), ([x, y], [torch.empty_like(x), x.view(6, 4)])):
        with pytest.raises(ValueError, match="shares memory"):
            m.clip_grads(grads, 1.0, out=out)
    assert torch.equal(b, torch.ones_like(b))
    # read twice is no conflict, nor are neighbours or an input as its own output
    m.clip_grads([b, b], 1e9, out=[torch.empty_like(b), torch.empty_like(b)])
    m.clip_grads([b[:50], b[50:], b[:0]], 1e9)
    m.clip_grads([b[:50], b[50:]], 1e9, out=[b[:50], torch.empty(50, device="cuda")])
    assert torch.equal(x, torch.ones(4, 6, device="cuda"))


def test_clip_more_chunks_than_workgroups():
    """Enough elements for the workgroups to take several chunks each; odd ends, some tensors in place."""
    m = sco()
    sizes = [200_000_003, 8192 * 9000, 5, 1_000_001]
    grads = [torch.full((n,), 0.5, device="cuda", dtype=torch.bfloat16) for n in sizes]
    out = [grads[0], torch.zeros_like(grads[1]), grads[2], torch.zeros_like(grads[3])]
    norm = 0.5 * math.sqrt(sum(sizes))
    r = m.clip_grads(grads, norm / 2, out=out)
    assert r.norm.item() == pytest.approx(norm, rel=2 * U) and r.scale.item() == pytest.approx(0.5, rel=1e-6)
    for x in out:  # 0.25 but for the factor's last bits, which bfloat16 has none of
        assert (x == 0.25).all()
    assert (grads[1] == 0.5).all() and (grads[3] == 0.5).all()
    r = m.clip_grads([grads[1]], 1e9)  # not reached: as they are
    assert r.scale.item() == 1.0 and (grads[1] == 0.5).all()
    r = m.clip_grads([grads[1]], 1e9, out=[out[1]])
    assert torch.equal(out[1], grads[1])


@pytest.mark.parametrize("T,V,kind", [(128, 140001, "half"), (100, 170001, "none")])
def test_policy_few_tokens_many_logits(T, V, kind):
    """Few tokens' own products of logits and weights' gradient, with logits relative to their rows' references."""
    H = 72
    g = gen(67)
    h, W, tgt = _xent_case(g, T, V, H, torch.bfloat16)
    h[1::4] *= 40.0  # some out of their references' reach
    tgt = _mask(tgt, kind, V)
    ref = Tokens(h, W, tgt, torch.bfloat16)
    old, adv, refl, _ = _policy_inputs(g, ref, (0.2, 0.2))
    out = sco().policy_loss(h, W, tgt, old.cuda(), adv.cuda(), ref_logp=refl.cuda(), kl=0.02)
    loss, dloss, _, _, _, _, c, dc, _ = _policy_ref(ref, old, adv, refl, None, (0.2, 0.2), 0.02)
    within("loss", out.loss.cpu(), loss, dloss)
    dh, dW, tdh, tdW = ref.gradients(c, dc)
    within("dh", out.dh.cpu(), dh, tdh)
    within("dW", out.dW.cpu(), dW, tdW)


def test_many_logits_graph_replays():
    """Losses whose logits are relative to their rows' references, captured and replayed on other tokens."""
    m, g = sco(), gen(68)
    T, V, H = 640, 27000, 128
    h, W, tgt = _xent_case(g, T, V, H, torch.bfloat16)
    f = randn(g, T, std=0.3)
    starts = torch.tensor([0, 200, 380, 500, 640], device="cuda")

    def step():
        lp = m.token_logp(h, W, tgt)
        return [lp, *m.policy_loss(h, W, tgt, lp + f, f, ref_logp=lp - f, kl=0.1), *m.preference_loss(h, W, tgt, starts)]

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k, share in enumerate((0.5, 0.0, 1.0, 0.1)):
        h.copy_(randn(g, T, H, std=(0.1, 1.0, 0.3, 4.0)[k], dtype=torch.bfloat16))
        t = torch.randint(0, V, (T,), generator=g, device="cuda")
        tgt.copy_(torch.where(torch.rand(T, generator=g, device="cuda") < share, -1, t))
        want = [x.clone() for x in step()]
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, out):
            assert torch.equal(a, b), k


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("chunks", [1, 255, 256, 257, 1000, 1023, 1024, 1025, 2300])
def test_clip_by_number_of_partial_sums(chunks, dtype):
    """One call for norm and clipping, whose partial sums are added up in one way or the other, against the sum given."""
    m, g = sco(), gen(69)
    n = 8192 * chunks - 5
    grads = [randn(g, n - n // 3, dtype=dtype), randn(g, n // 3, dtype=dtype)] if chunks > 1 else [randn(g, n, dtype=dtype)]
    total = sum((x.to(F64) ** 2).sum() for x in grads)
    s = m.grad_sumsq(grads)
    # sums of 64 bits in other orders
    assert abs(s - total) <= 1e-12 * total
    out = [torch.empty_like(x) for x in grads]
    a, b = m.clip_grads(grads, 3.0, out=out), m.clip_grads(grads, 3.0, out=[torch.empty_like(x) for x in grads], sumsq=s)
    norm = total.sqrt()
    assert abs(a.norm.to(F64) - norm) <= (U + 1e-12) * norm and abs(b.norm.to(F64) - norm) <= (U + 1e-12) * norm
    scale = 3.0 / (norm + 1e-6)
    assert abs(a.scale.to(F64) - scale) <= (U + 1e-12) * scale
    for x, y, z in zip(grads, a.grads, b.grads):
        want = x.to(F64) * scale
        for got in (y, z):  # the factor's rounding, the product's, the output's
            assert ((got.to(F64) - want).abs() <= (HALF[dtype] + 3 * U) * want.abs() + TINY).all()
    assert torch.equal(a.norm, m.clip_grads(grads, 3.0, out=out).norm)


@pytest.mark.parametrize("T,V,H,kind", [(9001, 2000, 72, "half"), (20000, 1030, 40, "runs")])
def test_policy_many_tokens(T, V, H, kind):
    """More tokens than find their rows in one launch with the operand, with logits relative to their rows' references."""
    g = gen(70)
    h, W, tgt = _xent_case(g, T, V, H, torch.bfloat16)
    tgt = _mask(tgt, kind, V)
    ref = Tokens(h, W, tgt, torch.bfloat16)
    old, adv, refl, _ = _policy_inputs(g, ref, (0.2, 0.2))
    out = sco().policy_loss(h, W, tgt, old.cuda(), adv.cuda(), ref_logp=refl.cuda(), kl=0.02)
    loss, dloss, total, dtotal, _, _, c, dc, _ = _policy_ref(ref, old, adv, refl, None, (0.2, 0.2), 0.02)
    within("logp", out.logp.cpu(), ref.logp, ref.dlogp)
    within("loss", out.loss.cpu(), loss, dloss)
    within("total", out.total.cpu(), total, dtotal)
    dh, dW, tdh, tdW = ref.gradients(c, dc)
    within("dh", out.dh.cpu(), dh, tdh)
    within("dW", out.dW.cpu(), dW, tdW)
    for off in ((out.dh.cpu().to(F64) - dh).norm() / dh.norm(), (out.dW.cpu().to(F64) - dW).norm() / dW.norm()):
        assert off <= 4 * HALF[torch.bfloat16], off
