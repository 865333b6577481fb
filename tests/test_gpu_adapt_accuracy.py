"""The gradients of the policy and preference losses in the mean: how far they are off in the norm, and along
themselves, against 64 bits.  The elementwise bounds count every rounding at its worst and would not see one more.

bfloat16: the roundings that the operators say they make are made here too, of the values in 64 bits: of softmax -
onehot, of the rows of h times the tokens' factors, each factor times what makes the target's entry exact, and of the
results.  What this is off in the norm, the operators may be, and a quarter more: one more rounding of dW or dh would
be sqrt(3 / 2) or sqrt(2) times as much.  Along the gradient itself the roundings average out: over the elements, and
the rows' factors (each off by HALF / sqrt(3) in the root of the mean square) over the n tokens that have weight; four
standard deviations are allowed.

float32: a logit s is off by its operands (2^-22 of each, at most 2 x 4 U in the root of the mean square of s) and by
the sums of H terms in three products, 32 at a time (sqrt(3 H / 32) U); so is what the logits make, once through
the exponentials and once through the coefficients.  The products with d add the sums of their V or T terms in six
products, and 8 U for what is left out and stored.  Twice that is allowed."""
import math

import pytest
import torch

from tests.gpu_harness import say
from tests.test_gpu_adapt import Tokens, _mask, _policy_inputs, _policy_ref
from tests.test_gpu_train import DT, F64, HALF, U, _xent_case, gen, randn, sco

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def near(name, got, want, bound, along):
    got, want = got.cpu().to(F64), want
    off = ((got - want).norm() / want.norm()).item()
    bias = abs(((got - want) * want).sum().item()) / (want * want).sum().item()
    say(f"  {name}: off {off:.3e} of {bound:.3e}, along {bias:.3e} of {along:.3e}")
    assert off <= bound and bias <= along, (name, off, bound, bias, along)


def rounded(ref, c, dh, dW):
    """How far dh and dW are off in the norm by bfloat16's roundings alone."""
    b16 = lambda x: x.to(torch.bfloat16).to(F64)
    unit = ref.p.clone().scatter_add_(1, ref.at, -torch.ones(ref.T, 1, dtype=F64))
    d = b16(unit)
    q, r = unit.gather(1, ref.at), d.gather(1, ref.at)
    f = c[:, None] * torch.where(r != 0, q / r, 1.0)
    return [((b16(x) - want).norm() / want.norm()).item()
            for x, want in (((d * f) @ ref.W, dh), (d.t() @ b16(ref.h * f), dW))]


def bounds(dtype, ref, c, dh, dW):
    """(norm, along) of dh and of dW."""
    if dtype == torch.bfloat16:
        weight = (c * c)[ref.ok]
        n = (weight.sum() ** 2 / (weight * weight).sum()).item()  # tokens that the norm is made of
        return [(1.25 * off, 4 * HALF[dtype] / math.sqrt(3 * n)) for off in rounded(ref, c, dh, dW)]
    s = (ref.h[ref.ok] @ ref.W.t()).square().mean().sqrt().item()
    logits = 2 * (8 + math.sqrt(3 * ref.h.shape[1] / 32)) * U * (1 + s)
    off = [2 * (logits + (math.sqrt(6 * k / 32) + 8) * U) for k in (ref.V, ref.T)]
    return [(x, x) for x in off]


SIZES = [(300, 3000, 520, "runs"), (120, 20000, 264, "none"), (700, 24100, 72, "runs"), (1500, 5000, 1032, "half"),
         (2000, 9000, 136, "none")]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("limit", [0, 1 << 24])
@pytest.mark.parametrize("T,V,H,kind", SIZES)
def test_policy_gradients_in_the_mean(T, V, H, kind, limit, dtype):
    say(f"case: policy in the mean T {T} V {V} H {H} {kind} limit {limit} {dtype}")
    g = gen(101)
    h, W, tgt = _xent_case(g, T, V, H, dtype)
    tgt = _mask(tgt, kind, V)
    ref = Tokens(h, W, tgt, dtype)
    old, adv, refl, _ = _policy_inputs(g, ref, (0.2, 0.2))
    out = sco().policy_loss(h, W, tgt, old.cuda(), adv.cuda(), ref_logp=refl.cuda(), kl=0.02, limit=limit)
    c = _policy_ref(ref, old, adv, refl, None, (0.2, 0.2), 0.02)[6]
    dh, dW = ref.gradients(c, torch.zeros_like(c))[:2]
    (bh, ah), (bw, aw) = bounds(dtype, ref, c, dh, dW)
    near("dh", out.dh, dh, bh, ah)
    near("dW", out.dW, dW, bw, aw)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("average", [False, True])
@pytest.mark.parametrize("T,V,H,kind", SIZES)
def test_preference_gradients_in_the_mean(T, V, H, kind, average, dtype):
    """All tokens of a sequence have one coefficient: a rounding of it would be the same in all of them."""
    say(f"case: preference in the mean T {T} V {V} H {H} {kind} average {average} {dtype}")
    g = gen(102)
    h, W, tgt = _xent_case(g, T, V, H, dtype)
    tgt = _mask(tgt, kind, V)
    ref = Tokens(h, W, tgt, dtype)
    starts = [0, T // 4, T // 2, T - T // 3, T]
    refl = (ref.logp + randn(g, T, std=0.1).cpu()).float()
    beta = 0.5
    out = sco().preference_loss(h, W, tgt, torch.tensor(starts, device="cuda"), ref_logp=refl.cuda(), beta=beta,
                                average=average)
    x = torch.where(ref.ok, ref.logp - refl.to(F64), 0.0)
    c = torch.zeros(T, dtype=F64)
    for p in range(2):
        part = [slice(starts[2 * p + k], starts[2 * p + k + 1]) for k in range(2)]
        share = [1 / max(1, int(ref.ok[s].sum())) if average else 1.0 for s in part]
        z = beta * (share[0] * x[part[0]].sum() - share[1] * x[part[1]].sum())
        for k in range(2):
            c[part[k]] = (1 - 2 * k) * beta / 2 * share[k] * torch.sigmoid(-z)
    c = torch.where(ref.ok, c, 0.0)
    dh, dW = ref.gradients(c, torch.zeros_like(c))[:2]
    (bh, ah), (bw, aw) = bounds(dtype, ref, c, dh, dW)
    near("dh", out.dh, dh, bh, ah)
    near("dW", out.dW, dW, bw, aw)
