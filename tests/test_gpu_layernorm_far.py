"""Layer norm's gradient of float32 rows far from 0, from h and the row's float32 mean, against the gradient of the
norm in 64 bits: half a step of the mean is much of such a row's deviation, and shifts all of it.  The tolerances
count roundings, as in tests/test_gpu_train.py."""
import pytest
import torch

from tests.gpu_harness import say
from tests.test_gpu_train import F64, TINY, U, gen, randn, sco, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("base,std", [(100.0, 1e-3), (-3000.0, 0.02), (1e6, 1.0), (0.1, 1e-6)])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,H", [(1, 64), (5, 20), (130, 257), (600, 1000), (40, 2048), (9, 4100), (3, 8192), (2, 16383)])
def test_gradient_of_rows_far_from_zero(T, H, residual, base, std):
    say(f"case: layernorm far T {T} H {H} base {base} std {std} residual {residual}")
    m, g = sco(), gen(91)
    x = randn(g, T, H, std=std) + base * (1 + 0.3 * randn(g, T, 1))
    r = randn(g, T, H, std=std) if residual else None
    gain, dy, dh = randn(g, H), randn(g, T, H), randn(g, T, H)
    eps = 2.0 ** -30
    out = m.layernorm(x, gain, residual=r, eps=eps, keep=False)
    dx, dgain, dbias = m.layernorm_grad(dy, gain, out.rstd, h=out.h, mean=out.mean, dh=dh)
    h = x.to(F64) + (0 if r is None else r.to(F64))
    mu = h.mean(1, keepdim=True)
    rs = 1 / ((h - mu).square().mean(1, keepdim=True) + eps).sqrt()
    n, a = (h - mu) * rs, dy.to(F64) * gain.to(F64)
    c0, c1 = a.mean(1, keepdim=True), (a * n).mean(1, keepdim=True)
    # n: h's own rounding where it is a sum, the difference (exact without a rounding of h), the factor and its
    # product, and the mean of what they make, a sum of 64 + 8 + 3 roundings of terms of n and of the mean's rounding
    terms, shift = (64 + 8 + 3) * U, U * mu.abs() * rs
    own = (1 if residual else 0) * U * h.abs() * rs
    size = n.abs() + shift + own
    en = 2 * own + 4 * U * size + own.mean(1, keepdim=True) + terms * size.mean(1, keepdim=True)
    dc0 = terms * a.abs().mean(1, keepdim=True)
    dc1 = (terms * a.abs() * size + a.abs() * en).mean(1, keepdim=True) + 2 * U * shift * c0.abs() + shift * dc0
    want = dh.to(F64) + rs * (a - c0 - n * c1)
    part = rs * (a.abs() + c0.abs() + n.abs() * c1.abs())
    more = rs * (dc0 + n.abs() * dc1 + en * (c1.abs() + dc1))
    within("dx", dx, want, U * want.abs() + 8 * U * (part + dh.to(F64).abs()) + more + TINY)
    d = dy.to(F64)
    within("dgain", dgain, (d * n).sum(0), ((T + 40) * U * (d * n).abs() + d.abs() * en).sum(0))
    within("dbias", dbias, d.sum(0), (T + 40) * U * d.abs().sum(0))


def test_a_mean_of_the_callers_own_is_taken_as_it_is():
    """A mean that is not the row's is the formula's (no rounding makes it 1e-4 of itself off)."""
    m, g = sco(), gen(92)
    T, H = 50, 300
    h, dy, gain = randn(g, T, H) + 5.0, randn(g, T, H), randn(g, H)
    mean, rstd = h.mean(1) * (1 + 1e-4), torch.ones(T, device="cuda")
    _, dgain, _ = m.layernorm_grad(dy, gain, rstd, h=h, mean=mean)
    n = h.to(F64) - mean.to(F64)[:, None]
    d = dy.to(F64)
    within("dgain", dgain, (d * n).sum(0), ((T + 40) * U * (d * n).abs() + 2 * U * (d * n).abs()).sum(0))
