"""GPU tests of how exact the training-step operators are: what is rounded to fewer bits, how often,
and which values survive.

U = 2^-24 is half a step of float32, H16 = 2^-8 of bfloat16, relative to the value."""
import math

import numpy as np
import pytest
import torch

from tests.gpu_harness import say
from tests.test_train_bounds import rms, rms_bound

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
H16 = 2.0 ** -8
F64 = torch.float64


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def sco():
    import spectral_correction_optimizer_amd as m
    return m


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


# ---- cross entropy: the logit gradients ----------------------------------------------------
# With h the identity, the logits are W's columns and dW[v][t] is token t's gradient of logit v over
# the count, a power of two: the gradient product adds nothing but zeros to it, so dW shows d itself.

# kept: one piece; limit 1: in pieces, each recomputed; T of each tile shape
@pytest.mark.parametrize("limit", [0, 1])
@pytest.mark.parametrize("T,V", [(1, 5000), (64, 3001), (256, 2000)])
def test_xent_rounds_each_logit_gradient_once(T, V, limit):
    """Half a step of bfloat16, and at most a quarter of that again for the exponential that is kept
    between the passes."""
    say(f"case: xent logit gradients T {T} V {V} limit {limit}")
    g = gen(1)
    W = (torch.randn(V, T, generator=g, device="cuda") * 1.5).bfloat16()
    tgt = torch.randint(0, V, (T,), generator=g, device="cuda")
    out = sco().xent(torch.eye(T, dtype=torch.bfloat16, device="cuda"), W, tgt, limit=limit)
    s = W.to(F64)
    lse = torch.logsumexp(s, 0)
    p = torch.exp(s - lse)
    ref = p.clone()
    at = torch.arange(T, device="cuda")
    ref[tgt, at] -= 1
    got = out.dW.to(F64) * T
    # float32: log-sum-exp, difference, exponential
    f32 = (8 * s.abs().amax(0) + 4 * lse.abs() + 400 + V / 64 + 32) * U
    rel = H16 * (1 if limit else 1.25) + H16 ** 2 + 2 * f32
    tol = p * rel
    tol[tgt, at] = ref[tgt, at].abs() * H16 + 2 * f32 * p[tgt, at] + 4 * U
    bad = (got - ref).abs() > tol
    assert not bad.any(), (int(bad.sum()), float(((got - ref).abs() / tol).max()))


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_xent_kept_exponentials_of_far_logits(sign):
    """All logits of a token alike and beyond 2^24, where a tile's reference in powers of two lies a
    whole number below the largest exponent unless it is raised: the probabilities stay 1 / V within
    what float32 resolves of such logits."""
    V, T = 200, 64
    log2e = np.float32(1.44269504088896340736)
    x = torch.arange(129, 256, dtype=F64) * 2.0 ** 18  # bfloat16 values from 2^25 on
    x = (sign * x).numpy().astype(np.float32)
    ref = np.ceil((x * log2e).astype(np.float32)).astype(np.float64)
    above = x.astype(np.float64) * np.float64(log2e) - ref
    x = x[above >= 1]
    assert x.size >= 16
    x = torch.from_numpy(np.resize(x, T)).cuda()
    W = x[None, :].expand(V, T).bfloat16().contiguous()
    assert torch.equal(W[0].float(), x)
    out = sco().xent(torch.eye(T, dtype=torch.bfloat16, device="cuda"), W, torch.zeros(T, dtype=torch.long, device="cuda"))
    got = out.dW[1:].to(F64) * T
    assert (got > 0).all()
    off = (got * V).log().abs()
    assert (off <= 8 * x.abs().to(F64) * U + H16 * 2).all(), float(off.max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("limit", [0, 1])
def test_xent_sums_of_the_largest_states(limit, dtype):
    """States of 2^127: the mean's gradients are within float32's range, the plain sums over the tokens
    are not."""
    from tests.test_gpu_train import _xent_check, _xent_ref
    T, V, H = 30, 300, 8
    say(f"case: xent sums of the largest states limit {limit} {dtype}")
    g = gen(4)
    h = torch.randn(T, H, generator=g, device="cuda")
    W = torch.randn(V, H, generator=g, device="cuda")
    h[:, 0] = 2.0 ** 127
    W[:, 0] = torch.randint(-8, 9, (V,), generator=g, device="cuda") * 2.0 ** -125
    h, W = h.to(dtype), W.to(dtype)
    tgt = torch.randint(0, 5, (T,), generator=g, device="cuda")
    ref, tol = _xent_ref(h, W, tgt, dtype)
    assert ref[3].abs().max() * T > 2.0 ** 128 > ref[3].abs().max()
    _xent_check(sco().xent(h, W, tgt, limit=limit), ref, tol)


# ---- float32 operands that bfloat16 cannot hold ---------------------------------------------

MOST = float(np.finfo(np.float32).max)
FAR = [math.inf, -math.inf, math.nan, MOST, -MOST, float.fromhex("0x1.ffp127"), -float.fromhex("0x1.ff0002p127"),
       float.fromhex("0x1.fefffep127"), float.fromhex("0x1.fep127")]


def test_act_wgrad_keeps_infinities_and_the_largest_values():
    """float32's largest values round to infinity in bfloat16, where the operand's planes begin: the
    gradient of each output holds what the definition gives, and an infinity stays one."""
    T, H = 40, 72
    N = len(FAR) + 3
    say(f"case: act_wgrad far values T {T} N {N} H {H}")
    g = gen(2)
    dy = torch.randn(T, N, generator=g, device="cuda")
    for i, x in enumerate(FAR):
        dy[7 * i % T, i] = x
    kept = sco().act_pack(torch.randn(T, H, generator=g, device="cuda") * 2.0 ** -12)
    n = sco().act_unpack(kept, torch.float32).cpu().to(F64)
    d64 = dy.cpu().to(F64)
    ref, mag = d64.t() @ n, d64.abs().t() @ n.abs()
    got = sco().act_wgrad(dy, kept).cpu().to(F64)
    assert torch.equal(got.isnan(), ref.isnan())
    assert torch.equal(got.isinf(), ref.isinf()) and torch.equal(got[ref.isinf()], ref[ref.isinf()])
    fin = ref.isfinite()
    assert fin[3:].all()
    # three products of T terms, two half steps a term, and the store
    tol = ref.abs() * 2 * U + (3 * T + 64) * 2 * U * mag
    assert ((got - ref).abs() <= tol)[fin].all()


@pytest.mark.parametrize("limit", [0, 1])
def test_xent_with_the_largest_states(limit):
    """Float32 states next to the largest number, against weights that bring the logits back."""
    from tests.test_gpu_train import _xent_check, _xent_ref
    T, V, H = 30, 300, 8
    say(f"case: xent largest states limit {limit}")
    g = gen(3)
    h = torch.randn(T, H, generator=g, device="cuda")
    W = torch.randn(V, H, generator=g, device="cuda")
    big = [x for x in FAR if math.isfinite(x)]
    h[:, 0] = torch.tensor([big[t % len(big)] for t in range(T)], device="cuda")
    W[:, 0] = torch.randint(-8, 9, (V,), generator=g, device="cuda") * 2.0 ** -125
    tgt = torch.randint(0, V, (T,), generator=g, device="cuda")
    ref, tol = _xent_ref(h, W, tgt, torch.float32)
    _xent_check(sco().xent(h, W, tgt, limit=limit), ref, tol)


# ---- float32 products: the error's norm -----------------------------------------------------
# (what a missing plane would do to it: tests/test_train_bounds.py)

@pytest.mark.parametrize("T,N,H", [(2, 96, 200), (63, 65, 33), (1999, 96, 200)])
def test_act_wgrad_has_the_accuracy_of_float32(T, N, H):
    say(f"case: act_wgrad error T {T} N {N} H {H}")
    g = gen(5)
    dy = torch.randn(T, N, generator=g, device="cuda")
    kept = sco().act_pack(torch.randn(T, H, generator=g, device="cuda"))
    n = sco().act_unpack(kept, torch.float32).cpu().to(F64)
    off = rms(sco().act_wgrad(dy, kept).cpu(), dy.cpu().to(F64).t() @ n)
    assert off <= rms_bound(3, T), off / U


@pytest.mark.parametrize("limit", [0, 1])
def test_xent_logits_have_the_accuracy_of_float32(limit):
    """Two words, one of them all zeros, and targets on the lesser logit: the loss is the other
    logit's magnitude."""
    T, H = 300, 520
    g = gen(6)
    h = torch.randn(T, H, generator=g, device="cuda") * 20
    W = torch.randn(2, H, generator=g, device="cuda") * 20
    W[1] = 0
    x = h.cpu().to(F64) @ W[0].cpu().to(F64)
    out = sco().xent(h, W, (x > 0).long().cuda(), limit=limit)
    ref = x.abs() + torch.log1p(torch.exp(-x.abs()))
    off = rms(out.loss.cpu(), ref)
    assert off <= rms_bound(6, H), off / U


@pytest.mark.parametrize("limit", [0, 1])
def test_xent_gradients_have_the_accuracy_of_float32(limit):
    """Logits and log-sum-exp below 8: they and their difference are off by at most 14 U in the mean."""
    T, V, H = 300, 700, 520
    g = gen(7)
    h = torch.randn(T, H, generator=g, device="cuda") / math.sqrt(H)
    W = torch.randn(V, H, generator=g, device="cuda") * 0.5
    tgt = torch.randint(0, V, (T,), generator=g, device="cuda")
    out = sco().xent(h, W, tgt, limit=limit)
    h, W, at = h.cpu().to(F64), W.cpu().to(F64), torch.arange(T)
    s = h @ W.t()
    lse = torch.logsumexp(s, 1, keepdim=True)
    assert s.abs().max() < 8 and lse.abs().max() < 8
    d = torch.exp(s - lse)
    d[at, tgt.cpu()] -= 1
    for name, got, ref, K in (("dh", out.dh, d @ W / T, V), ("dW", out.dW, d.t() @ h / T, T)):
        off = rms(got.cpu(), ref)
        assert off <= rms_bound(6, K, 14), (name, off / U)


# ---- residual norm: the 8-bit values are those of the rows in 64 bits -------------------------

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", [(4096, 1000), (2048, 2048), (300, 8191), (100, 16384)])
def test_rmsnorm_picks_the_steps_of_64_bits(T, H, dtype):
    """Every element of millions, but for those within 1e-10 of the border of two steps (of which
    float32 rows missed a few in a million), and the statistics to a float32's rounding."""
    from tests.test_gpu_train import pow2
    say(f"case: rmsnorm steps T {T} H {H} {dtype}")
    g = gen(8)
    x = (torch.randn(T, H, generator=g, device="cuda") * 0.5).to(dtype)
    r = torch.randn(T, H, generator=g, device="cuda").to(dtype)
    gain = torch.randn(H, generator=g, device="cuda").to(dtype)
    eps = 2.0 ** -17
    out = sco().rmsnorm(x, gain, residual=r, eps=eps)
    h = x.to(F64) + r.to(F64)
    rstd = 1 / (h.square().mean(1) + eps).sqrt()
    assert ((out.rstd.to(F64) - rstd).abs() <= U * (1 + 1e-6) * rstd).all()
    n = h * rstd[:, None]
    half = U if dtype == torch.float32 else H16
    y = n * gain.to(F64)
    assert ((out.y.to(F64) - y).abs() <= (half + 2 * U) * (1 + 1e-6) * y.abs()).all()
    nb = -(-H // 32)
    p = torch.zeros(T, nb * 32, dtype=F64, device="cuda")
    p[:, :H] = n
    p = p.reshape(T, nb, 32)
    amax = p.abs().amax(2)
    m, E = torch.frexp(amax)  # amax = m 2^E, m in [0.5, 1)
    clear = ((m - 0.5).abs() > 1e-10) & ((1 - m).abs() > 1e-10)
    assert clear.float().mean() > 0.999
    assert torch.equal(out.kept.e[clear].int(), (E + 126)[clear].int())
    steps = p * pow2(7 - E)[:, :, None]
    border = (steps - steps.floor() - 0.5).abs() < 1e-10
    want = steps.round().clamp(-127, 127)
    q = torch.zeros(T, nb * 32, device="cuda", dtype=F64)
    q[:, :H] = out.kept.q.to(F64)
    same = (q.reshape(T, nb, 32) == want) | border | ~clear[:, :, None]
    assert border.sum() < 100 and same.all(), int((~same).sum())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("limit", [0, 1])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_xent_states_that_are_not_finite(value, limit, dtype):
    """A counted token's: its loss, its row of dh, the mean and dW are NaN, the other rows are not.  A
    token that is not counted: nothing is."""
    T, V, H = 70, 300, 64
    g = gen(9)
    h = torch.randn(T, H, generator=g, device="cuda").to(dtype)
    W = torch.randn(V, H, generator=g, device="cuda").to(dtype)
    tgt = torch.randint(0, V, (T,), generator=g, device="cuda")
    h[5, 7] = value
    out = sco().xent(h, W, tgt, limit=limit)
    rest = torch.arange(T, device="cuda") != 5
    assert out.loss[5].isnan() and out.mean.isnan() and out.dh[5].isnan().all() and out.dW.isnan().all()
    assert out.loss[rest].isfinite().all() and out.dh[rest].isfinite().all()
    tgt[5] = V
    out = sco().xent(h, W, tgt, limit=limit)
    assert all(t.isfinite().all() for t in out)
