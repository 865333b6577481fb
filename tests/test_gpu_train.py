"""GPU parity of the training-step operators (embedding, residual norm with its 8-bit
checkpoint, the gradients that read it, large-vocabulary cross entropy) against their
definitions in 64 bits.

Tolerances count roundings.  U = 2^-24 is half a step of float32, H16 = 2^-8 of bfloat16
(relative to the value).  A float32 sum of n terms is off by at most n U times the sum of
the terms' magnitudes; matrix-core sums are counted at 2 U a term, as their internal
rounding need not be to nearest."""
import math

import numpy as np
import pytest
import torch

from tests.gpu_harness import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TINY = 2.0 ** -126
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
F64 = torch.float64
DT = [torch.bfloat16, torch.float32]


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


def randn(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def pow2(e):
    """2^e in 64 bits, exact (the device's powers need not be)."""
    return torch.from_numpy(np.ldexp(1.0, e.cpu().to(torch.int32).numpy())).to(e.device)


def within(name, got, ref, tol):
    """Elementwise |got - ref| <= tol, NaN only where the reference has it."""
    got = got.to(F64)
    assert torch.equal(got.isnan(), ref.isnan()), f"{name}: NaN in other places"
    d = (got - ref).abs()
    bad = (d > tol) & ~ref.isnan() & (got != ref)
    if bad.any():
        i = bad.nonzero()[0].tolist()
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} outside, first at {i}: got "
                             f"{got[tuple(i)].item()} want {ref[tuple(i)].item()} tol {tol[tuple(i)].item()}")


# ---- embedding ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T,V,H", [(0, 5, 8), (1, 1, 1), (7, 11, 3), (33, 100, 64), (5, 17, 257), (300, 1000, 1001)])
def test_embed(T, V, H, dtype):
    say(f"case: embed T {T} V {V} H {H} {dtype}")
    g = gen(1)
    table = randn(g, V, H, dtype=dtype)
    ids = torch.randint(-2, V + 2, (T,), generator=g, device="cuda")
    scale = 1.7
    out = sco().embed(table, ids, scale=scale)
    ref = table.to(F64)[ids.clamp(0, V - 1)] * scale
    ref[(ids < 0) | (ids >= V)] = 0
    within("out", out, ref, ref.abs() * (HALF[dtype] + 3 * U))


def _embed_grad_ref(dy, ids, V, scale):
    ok = (ids >= 0) & (ids < V)
    ref = torch.zeros(V, dy.shape[1], dtype=F64, device="cuda")
    mag = torch.zeros_like(ref)
    ref.index_add_(0, ids[ok], dy[ok].to(F64))
    mag.index_add_(0, ids[ok], dy[ok].to(F64).abs())
    n = torch.bincount(ids[ok], minlength=V).to(F64)[:, None]
    return ref * scale, mag * scale, n


# rows within one stretch of 32 sorted tokens, across two, across many (one id only), all
# tokens ignored, fewer tokens than a stretch, more than one block of 1024 tokens, ids of
# one bin and of many (V > 512), odd H, H over one slab of 512 columns
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T,V,H,kind", [(0, 3, 8, "uniform"), (1, 1, 1, "uniform"), (31, 4, 5, "uniform"),
                                        (100, 7, 64, "uniform"), (200, 3, 513, "one"), (64, 50, 33, "ignored"),
                                        (3000, 700, 40, "zipf"), (70000, 5000, 9, "zipf"), (2500, 20000, 1001, "zipf"),
                                        (4096, 131072, 16, "zipf"), (70000, 600, 8, "one")])
def test_embed_grad(T, V, H, kind, dtype):
    say(f"case: embed_grad T {T} V {V} H {H} {kind} {dtype}")
    g = gen(2)
    dy = randn(g, T, H, dtype=dtype)
    if kind == "uniform":
        ids = torch.randint(-1, V + 1, (T,), generator=g, device="cuda")
    elif kind == "one":
        ids = torch.full((T,), V - 1, device="cuda")
    elif kind == "ignored":
        ids = torch.where(torch.arange(T, device="cuda") % 2 == 0, -1, V)
    else:
        u = torch.rand(T, generator=g, device="cuda", dtype=F64)
        ids = ((torch.exp(u * math.log(V + 1)) - 1).long() * 7919) % V
    scale = 0.75  # exact in float32
    dW = sco().embed_grad(dy, ids, V, scale=scale)
    ref, mag, n = _embed_grad_ref(dy, ids, V, scale)
    within("dW", dW, ref, ref.abs() * (HALF[dtype] + U) + n * U * mag)
    # the same bits on every run
    assert torch.equal(dW, sco().embed_grad(dy, ids, V, scale=scale))


def test_embed_grad_is_the_gradient_of_embed():
    """Differences of <embed(table), dy> along random directions."""
    g = gen(3)
    V, H, T = 40, 24, 90
    table = randn(g, V, H)
    ids = torch.randint(-1, V, (T,), generator=g, device="cuda")
    dy, d = randn(g, T, H), randn(g, V, H)
    dW = sco().embed_grad(dy, ids, V, scale=3.0)
    f = [(sco().embed(table + s * d, ids, scale=3.0).to(F64) * dy.to(F64)).sum() for s in (0.5, -0.5)]
    # linear in the table: the difference is exact up to the roundings of table +- d / 2 and of the rows
    mag = (sco().embed(table.abs() + d.abs(), ids, scale=3.0).to(F64) * dy.abs().to(F64)).sum()
    slack = 8 * U * mag + 100 * U * (dW.abs().to(F64) * d.abs().to(F64)).sum()
    assert abs((f[0] - f[1]) - (dW.to(F64) * d.to(F64)).sum()) <= slack


# ---- 8-bit blocks ------------------------------------------------------------------------

def _pack_ref(x):
    """q, e of float64 rows that hold float32 values."""
    T, H = x.shape
    nb = -(-H // 32)
    p = torch.zeros(T, nb * 32, dtype=F64, device=x.device)
    p[:, :H] = x
    p = p.reshape(T, nb, 32)
    finite = p.isfinite().all(2)
    amax = torch.where(finite, p.abs().amax(2), torch.ones((), dtype=F64, device=x.device))
    E = (torch.frexp(amax)[1] - 1).clamp(min=-120)
    E = torch.where(amax == 0, -120, E)
    q = torch.round(p * pow2(6 - E)[:, :, None]).clamp(-127, 127)
    q = torch.where(finite[:, :, None], q, torch.zeros_like(q)).reshape(T, nb * 32)[:, :H]
    return q.to(torch.int8), torch.where(finite, E + 127, 255).to(torch.uint8)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T,H", [(0, 8), (1, 1), (3, 31), (4, 32), (5, 33), (40, 257), (7, 4100)])
def test_act_pack_unpack_exact(T, H, dtype):
    say(f"case: act_pack T {T} H {H} {dtype}")
    g = gen(4)
    x = randn(g, T, H) * torch.exp2(torch.randint(-130, 120, (T, 1), generator=g, device="cuda").float())
    x = x.to(dtype)
    if T > 2:
        x[0].zero_()
        x[1, 0] = math.inf
        x[2, H - 1] = math.nan
    k = sco().act_pack(x)
    q, e = _pack_ref(x.to(F64))
    assert torch.equal(k.e, e)
    assert torch.equal(k.q, q)
    for out in DT:
        y = sco().act_unpack(k, out)
        step = torch.where(e == 255, math.nan, pow2(e.to(torch.int32) - 133)).repeat_interleave(32, 1)[:, :H]
        ref = q.to(F64) * step
        assert torch.equal(y.to(F64).nan_to_num(7), ref.nan_to_num(7))


# ---- residual norm -----------------------------------------------------------------------

NORM_SIZES = [(1, 1), (3, 5), (9, 64), (130, 257), (6, 512), (5, 1000), (7, 2048), (4, 2051), (3, 4100), (2, 8192),
              (2, 16384), (1, 16383)]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T,H", NORM_SIZES)
def test_rmsnorm(T, H, dtype):
    say(f"case: rmsnorm T {T} H {H} {dtype}")
    g = gen(5)
    x, r = randn(g, T, H, dtype=dtype, std=0.5), randn(g, T, H, dtype=dtype)
    gain = randn(g, H, dtype=dtype)
    if T > 2:
        x[0].zero_()
        r[0].zero_()  # rstd = 1 / sqrt(eps)
        r[1] *= 1e4
    eps = 2.0 ** -17  # exact in float32
    out = sco().rmsnorm(x, gain, residual=r, eps=eps)
    h = x.to(F64) + r.to(F64)
    within("h", out.h, h, h.abs() * (HALF[dtype] + 2 * U))
    # squares: each h twice U, the product, at most 64 + 8 additions; / H, + eps: 2 more; half of it
    # in the root, then the root and the quotient
    drs = (0.5 * (2 + 1 + 72 + 2) + 2) * U
    rstd = 1 / (h.square().mean(1) + eps).sqrt()
    within("rstd", out.rstd, rstd, rstd * drs)
    n = h * rstd[:, None]
    dn = drs + 2 * U
    y = n * gain.to(F64)
    within("y", out.y, y, y.abs() * (HALF[dtype] + dn + 2 * U))
    # the checkpoint: E from the block's largest value within dn, each value half a step off,
    # a clipped one (beyond 127 steps) up to a whole one
    nb = -(-H // 32)
    e = out.kept.e.to(torch.int32) - 127
    p = torch.zeros(T, nb * 32, dtype=F64, device="cuda")
    p[:, :H] = n
    amax = p.reshape(T, nb, 32).abs().amax(2)
    assert ((pow2(e) <= amax * (1 + dn)) | (e == -120)).all()
    assert (pow2(e + 1) > amax * (1 - dn)).all()
    step = pow2(e - 6).repeat_interleave(32, 1)[:, :H]
    got = sco().act_unpack(out.kept, torch.float32)
    clip = out.kept.q.abs() == 127
    within("kept", got, n, torch.where(clip, 1.0, 0.5) * step + dn * n.abs())
    # without a residual, and without a checkpoint
    two = sco().rmsnorm(x, gain, eps=eps, keep=False)
    assert two.kept is None and two.h is x
    xs = x.to(F64)
    y = xs / (xs.square().mean(1, keepdim=True) + eps).sqrt() * gain.to(F64)
    within("y alone", two.y, y, y.abs() * (HALF[dtype] + dn + 2 * U))


def test_rmsnorm_nonfinite_rows_stay_apart():
    """A NaN or an infinity reaches its own row only; its checkpoint reads as NaN."""
    g = gen(6)
    x, gain = randn(g, 6, 100), randn(g, 100)
    x[1, 3] = math.nan
    x[4, 99] = math.inf
    out = sco().rmsnorm(x, gain)
    kept = sco().act_unpack(out.kept, torch.float32)
    for t in range(6):
        assert bool(out.y[t].isfinite().all()) == (t not in (1, 4))
        assert bool(kept[t].isfinite().all()) == (t not in (1, 4))
    assert kept[1].isnan().all()


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T,H", [(0, 40)] + NORM_SIZES + [(5000, 96)])
def test_rmsnorm_grad(T, H, dtype):
    say(f"case: rmsnorm_grad T {T} H {H} {dtype}")
    g = gen(7)
    dy, dh = randn(g, T, H, dtype=dtype), randn(g, T, H, dtype=dtype)
    gain = randn(g, H, dtype=dtype)
    rstd = torch.rand(T, generator=g, device="cuda") + 0.5
    kept = sco().act_pack(randn(g, T, H))
    dx, dgain = sco().rmsnorm_grad(dy, gain, rstd, kept, dh=dh)
    n = sco().act_unpack(kept, torch.float32).to(F64)
    a = dy.to(F64) * gain.to(F64)
    c = (a * n).sum(1, keepdim=True) / H
    dc = (64 + 8 + 3) * U * (a * n).abs().sum(1, keepdim=True) / H  # a row's sum and its two products
    rs = rstd.to(F64)[:, None]
    ref = dh.to(F64) + rs * (a - n * c)
    part = rs * (a.abs() + n.abs() * c.abs())
    within("dx", dx, ref, ref.abs() * HALF[dtype] + 4 * U * (part + dh.to(F64).abs()) + rs * n.abs() * dc)
    dg = (dy.to(F64) * n).sum(0)
    within("dgain", dgain, dg, (T + 40) * U * (dy.to(F64) * n).abs().sum(0))
    # without the gradient past the norm, and the same bits again
    dx0, dgain0 = sco().rmsnorm_grad(dy, gain, rstd, kept)
    ref = rs * (a - n * c)
    within("dx alone", dx0, ref, ref.abs() * HALF[dtype] + 4 * U * part + rs * n.abs() * dc)
    assert torch.equal(dgain, dgain0)


def test_rmsnorm_grad_against_differences():
    """The gradient of <y, dy> + <h, dh> by differences in 64 bits at the checkpoint's rows: the
    checkpoint is made exact (rows of few bits), so only the gradient's own roundings remain."""
    g = gen(8)
    T, H, eps = 6, 64, 0.0
    x = torch.randint(-64, 65, (T, H), generator=g, device="cuda").double()
    x[:, ::8] = 64.0
    rms = x.square().mean(1, keepdim=True).sqrt()
    n = x / rms  # q * 2^(E - 6) holds multiples of 1/64 of it, up to the row's scale
    scale = 2.0 ** -6
    kept = sco().act_pack((x * scale).float())
    assert torch.equal(sco().act_unpack(kept, torch.float32).double(), x * scale)
    # rows whose normalised form is x * scale exactly: gain and dy absorb the rest
    gain, dy, dh = randn(g, H), randn(g, T, H), randn(g, T, H)

    def f(z, gn):
        m = z.square().mean(1, keepdim=True)
        return (z / m.sqrt() * gn * dy.double()).sum() + (z * dh.double()).sum()

    # n_kept = s n with s = rms * scale: dx of the operator for rstd = s^2 / rms and dy / s:
    # a n_kept / H term: (dy g / s)(s n) = dy g n, times n_kept = s n and rstd: folded below
    s = rms * scale
    dys = (dy.double() * s).float()
    rstd = (1 / (rms * s)).float().reshape(T)
    z = x.clone()
    d = torch.randn(T, H, generator=g, device="cuda", dtype=F64)
    t = 1e-5
    num = (f(z + t * d, gain.double()) - f(z - t * d, gain.double())) / (2 * t)
    a = dy.double() * gain.double()
    want = dh.double() + (a - n * (a * n).mean(1, keepdim=True)) / rms
    # the definition against differences (64 bits, error of order t^2)
    assert abs((want * d).sum() - num) <= 1e-7 * (want * d).abs().sum()
    # the operator against the definition, with n_kept = s n: a' = a s, n' = s n gives
    # a' - n' mean(a' n') = s (a - s^2 n mean(a n)); rows with s = 1 would be the norm itself
    dx, _ = sco().rmsnorm_grad(dys, gain, rstd, kept, dh=dh)
    an = (a * n).mean(1, keepdim=True)
    ref = dh.double() + (a - n * s * s * an) / rms
    mag = dh.double().abs() + (a.abs() + n.abs() * s * s * (a * n).abs().mean(1, keepdim=True)) / rms
    within("dx", dx, ref, 90 * U * mag)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T,H", [(40, 1000), (700, 4100), (300, 2049), (9, 8191), (5, 9001), (64, 7)])
def test_norm_in_place(T, H, dtype):
    """The C entries allow h = x, h = residual, dx = dy and dx = dh, also for rows that end inside a
    group of eight."""
    say(f"case: in place T {T} H {H} {dtype}")
    m, g = sco(), gen(21)
    lib, dt, st = m.load_library(), m._DT[dtype], torch.cuda.current_stream().cuda_stream
    x, r, dy, dh = (randn(g, T, H, dtype=dtype) for _ in range(4))
    gain = randn(g, H, dtype=dtype)
    want = m.rmsnorm(x, gain, residual=r)
    for i in range(2):
        a = [x.clone(), r.clone()]
        y, rstd = torch.empty_like(x), torch.empty(T, device="cuda")
        assert lib.sc_rmsnorm(dt, a[0].data_ptr(), a[1].data_ptr(), gain.data_ptr(), 1e-5, T, H, a[i].data_ptr(),
                              y.data_ptr(), rstd.data_ptr(), None, None, st) == 0
        assert torch.equal(a[i], want.h) and torch.equal(y, want.y) and torch.equal(rstd, want.rstd)
    dx, dgain = m.rmsnorm_grad(dy, gain, want.rstd, want.kept, dh=dh)
    n = m._workspace_bytes("sc_rmsnorm_grad_workspace", T, H)
    for i in range(2):
        a = [dy.clone(), dh.clone()]
        dg, ws = torch.empty(H, device="cuda"), torch.empty(n, dtype=torch.uint8, device="cuda")
        assert lib.sc_rmsnorm_grad(dt, a[0].data_ptr(), gain.data_ptr(), want.rstd.data_ptr(), want.kept.q.data_ptr(),
                                   want.kept.e.data_ptr(), a[1].data_ptr(), T, H, a[i].data_ptr(), dg.data_ptr(),
                                   ws.data_ptr(), n, st) == 0
        assert torch.equal(a[i], dx) and torch.equal(dg, dgain)


# ---- weight gradient from the checkpoint -------------------------------------------------

@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T,N,H", [(0, 5, 9), (1, 1, 1), (2, 8, 64), (63, 65, 33), (64, 64, 64), (65, 128, 256),
                                   (100, 300, 257), (257, 264, 520), (1999, 96, 200), (5000, 40, 72), (700, 513, 1000)])
def test_act_wgrad(T, N, H, dtype):
    say(f"case: act_wgrad T {T} N {N} H {H} {dtype}")
    g = gen(9)
    dy = randn(g, T, N, dtype=dtype)
    gain = randn(g, H, dtype=dtype)
    kept = sco().act_pack(randn(g, T, H))
    n = sco().act_unpack(kept, torch.float32).cpu().to(F64)
    d64 = dy.cpu().to(F64)
    ref = (d64.t() @ n).cuda()
    mag = (d64.abs().t() @ n.abs()).cuda()
    terms = T * (1 if dtype == torch.bfloat16 else 3) + 64  # and the sum over splits
    dW = sco().act_wgrad(dy, kept, gain=gain)
    gn = gain.to(F64)
    within("dW", dW, ref * gn, (ref * gn).abs() * (HALF[dtype] + U) + terms * 2 * U * mag * gn.abs())
    dW1 = sco().act_wgrad(dy, kept)
    within("dW without gain", dW1, ref, ref.abs() * (HALF[dtype] + U) + terms * 2 * U * mag)
    assert torch.equal(dW, sco().act_wgrad(dy, kept, gain=gain))


def test_products_of_views_off_16_bytes():
    """Contiguous views that start off 16 bytes: the binding copies them."""
    g = gen(10)
    dy = randn(g, 33, 24, dtype=torch.bfloat16).reshape(-1)[24 * 3:].reshape(30, 24)
    dy = torch.cat([dy.reshape(-1)[:1], dy.reshape(-1)])[1:].reshape(30, 24)
    assert dy.data_ptr() % 16
    kept = sco().act_pack(randn(g, 30, 40))
    assert torch.equal(sco().act_wgrad(dy, kept), sco().act_wgrad(dy.clone(), kept))


# ---- cross entropy -----------------------------------------------------------------------

def _xent_ref(h, W, tgt, dtype):
    """Values in 64 bits and the bounds of their errors (on the CPU)."""
    h, W, tgt = h.cpu().to(F64), W.cpu().to(F64), tgt.cpu()
    (T, H), V = h.shape, W.shape[0]
    ok = (tgt >= 0) & (tgt < V)
    at = tgt.clamp(0, V - 1)[:, None]
    count = max(1, int(ok.sum()))
    h = torch.where(ok[:, None], h, torch.zeros((), dtype=F64))
    s, smag = h @ W.t(), h.abs() @ W.abs().t()
    b16 = dtype == torch.bfloat16
    # a logit: H terms (six products each in float32, and the planes' remainder)
    es = (smag * ((H + 64) * 2 * U if b16 else ((6 * (H + 64)) * 2 + 4) * U)).amax(1, keepdim=True)
    smax = s.abs().amax(1, keepdim=True)
    lse = torch.logsumexp(s, 1, keepdim=True)
    # exp and log of values of size |s|, sums of at most 256 + tiles positive terms
    dlse = es + (8 * smax + 4 * lse.abs() + 400 + V / 64 + 16) * U
    loss = torch.where(ok[:, None], lse - s.gather(1, at), torch.zeros((), dtype=F64))
    dloss = torch.where(ok[:, None], es + dlse + 4 * U * (smax + lse.abs()), torch.zeros((), dtype=F64))
    p = torch.exp(s - lse)
    d = p.clone().scatter_add_(1, at, -torch.ones_like(lse)) * ok[:, None]
    rel = torch.expm1(es + dlse + (8 * smax + 16) * U)
    ed = p * rel * ok[:, None]
    ed += (2 * HALF[dtype] * p if b16 else 4 * U * p) * ok[:, None]
    ed.scatter_(1, at, (p * rel).gather(1, at) + (HALF[dtype] if b16 else 2 * U) * d.abs().gather(1, at))
    ed = (ed + TINY) * ok[:, None]  # below the smallest normal number float32 may hold zero
    share = 1 / count
    dh, dW = d @ W * share, d.t() @ h * share
    terms = 1 if b16 else 6
    da, ha, wa = d.abs() + ed, h.abs(), W.abs()
    tdh = share * (ed @ wa + (terms * (V + 64) + 8) * 2 * U * (da @ wa)) + dh.abs() * (HALF[dtype] + 4 * U) + TINY
    tdW = share * (ed.t() @ ha + (terms * (T + 64) + 8) * 2 * U * (da.t() @ ha)) + dW.abs() * (HALF[dtype] + 4 * U) + TINY
    mean = loss.sum() / count
    return ([loss[:, 0], mean, dh, dW],
            [dloss[:, 0], dloss.sum() / count + 4 * U * mean.abs(), tdh, tdW])


def _xent_case(g, T, V, H, dtype, spread=1.0):
    W = randn(g, V, H, std=0.5)
    tgt = torch.randint(0, V, (T,), generator=g, device="cuda")
    h = randn(g, T, H) * spread / math.sqrt(H)
    lean = torch.rand(T, 1, generator=g, device="cuda") * 20 / H
    h = h + lean * W[tgt]
    return h.to(dtype), W.to(dtype), tgt


def _xent_check(out, ref, tol):
    for name, got, r, t in zip(("loss", "mean", "dh", "dW"), out, ref, tol):
        within(name, got.cpu(), r, t)


# one tile and many, ends inside a tile, rows and columns of one, T of each tile shape,
# operands that are copied (H % 8) and used in place
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T,V,H", [(1, 1, 1), (1, 2, 8), (2, 5, 20), (3, 130, 64), (65, 33, 257), (64, 1000, 72),
                                   (130, 2500, 136), (300, 700, 520), (1, 5001, 64), (513, 257, 96)])
def test_xent(T, V, H, dtype):
    say(f"case: xent T {T} V {V} H {H} {dtype}")
    g = gen(11)
    h, W, tgt = _xent_case(g, T, V, H, dtype)
    if T > 2:
        tgt[1] = -1
        tgt[2] = V
    out = sco().xent(h, W, tgt)
    ref, tol = _xent_ref(h, W, tgt, dtype)
    _xent_check(out, ref, tol)
    again = sco().xent(h, W, tgt)
    for a, b in zip(out, again):
        assert torch.equal(a, b)


# pieces: the vocabulary in 2 to 10 of them, the last one short
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T,V,H,limit", [(64, 1000, 72, 1), (130, 2500, 136, 1), (300, 700, 520, 300 << 10),
                                         (5, 513, 33, 1)])
def test_xent_in_pieces(T, V, H, limit, dtype):
    say(f"case: xent pieces T {T} V {V} H {H} limit {limit} {dtype}")
    g = gen(12)
    h, W, tgt = _xent_case(g, T, V, H, dtype)
    tgt[0] = -1
    ref, tol = _xent_ref(h, W, tgt, dtype)
    _xent_check(sco().xent(h, W, tgt, limit=limit), ref, tol)


@pytest.mark.parametrize("dtype", DT)
def test_xent_nothing_counted_and_no_token(dtype):
    g = gen(13)
    h, W, tgt = _xent_case(g, 70, 300, 64, dtype)
    out = sco().xent(h, W, torch.full_like(tgt, -1))
    for t in out:
        assert torch.count_nonzero(t).item() == 0
    out = sco().xent(h[:0], W, tgt[:0])
    assert out.loss.shape == (0,) and out.mean.item() == 0 and torch.count_nonzero(out.dW).item() == 0


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("limit", [0, 1])
def test_xent_far_logits(dtype, limit):
    """Logits of several hundred in either direction: no overflow, no empty sum."""
    g = gen(14)
    T, V, H = 40, 900, 64
    h, W, tgt = _xent_case(g, T, V, H, dtype, spread=2000.0)
    ref, tol = _xent_ref(h, W, tgt, dtype)
    assert ref[0].max() > 500
    _xent_check(sco().xent(h, W, tgt, limit=limit), ref, tol)


@pytest.mark.parametrize("dtype", DT)
def test_xent_nonfinite_tokens(dtype):
    """A token that is not counted reaches nothing, even with NaN states; a counted one with NaN
    states has a NaN loss and the others' losses stay."""
    g = gen(15)
    h, W, tgt = _xent_case(g, 80, 500, 64, dtype)
    tgt[7] = -1
    clean = sco().xent(h, W, tgt)
    bad = h.clone()
    bad[7] = math.nan
    out = sco().xent(bad, W, tgt)
    for a, b in zip(clean, out):
        assert torch.equal(a, b)
    bad[20, 5] = math.inf
    out = sco().xent(bad, W, tgt)
    assert out.loss[20].isnan() and out.mean.isnan()
    keep = torch.arange(80, device="cuda") != 20
    assert torch.equal(out.loss[keep], clean.loss[keep])


def test_xent_against_differences():
    """The float32 gradients of the mean loss against differences of the 64-bit loss."""
    g = gen(16)
    T, V, H = 50, 320, 48
    h, W, tgt = _xent_case(g, T, V, H, torch.float32)
    out = sco().xent(h, W, tgt)
    dhd, dWd = torch.randn(T, H, dtype=F64), torch.randn(V, H, dtype=F64)

    def f(a, b):
        s = a @ b.t()
        return (torch.logsumexp(s, 1) - s.gather(1, tgt.cpu()[:, None])[:, 0]).mean()

    h64, W64, t = h.cpu().to(F64), W.cpu().to(F64), 1e-5
    num = (f(h64 + t * dhd, W64 + t * dWd) - f(h64 - t * dhd, W64 - t * dWd)) / (2 * t)
    got = (out.dh.cpu().to(F64) * dhd).sum() + (out.dW.cpu().to(F64) * dWd).sum()
    _, tol = _xent_ref(h, W, tgt, torch.float32)
    slack = (tol[2] * dhd.abs()).sum() + (tol[3] * dWd.abs()).sum() + 1e-6 * abs(num)
    assert abs(got - num) <= slack


# ---- streams and graphs ------------------------------------------------------------------

def test_other_stream_and_graph_replays():
    """The operators on a stream of their own, and captured into a graph that is replayed on new
    inputs, give the eager results bit for bit."""
    m = sco()
    g = gen(17)
    V, H, T = 600, 128, 200
    table, gain = randn(g, V, H, dtype=torch.bfloat16), randn(g, H, dtype=torch.bfloat16)
    ids = torch.randint(-1, V, (T,), generator=g, device="cuda")
    tgt = torch.randint(-1, V, (T,), generator=g, device="cuda")

    def step():
        x = m.embed(table, ids, scale=2.0)
        r = m.rmsnorm(x, gain, residual=x)
        o = m.xent(r.y, table, tgt)
        dx, dgain = m.rmsnorm_grad(o.dh, gain, r.rstd, r.kept, dh=o.dh)
        dW = m.act_wgrad(o.dh, r.kept, gain=gain)
        return [r.h, r.y, o.loss, o.mean, o.dW, dx, dgain, dW, m.embed_grad(dx, ids, V, scale=2.0)]

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
        ids.copy_(torch.randint(-1, V, (T,), generator=g, device="cuda"))
        tgt.copy_(torch.randint(-1, V, (T,), generator=g, device="cuda"))
        want = [t.clone() for t in step()]
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, out):
            assert torch.equal(a, b), k


# ---- many tiles a workgroup ----------------------------------------------------------------

# more output tiles than workgroups run at once, each way of storing them: whole 256 x 256 tiles and
# cut ones (and in float32 the six plane products of each)
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T,N,H", [(130, 4400, 4104), (200, 8192, 2304)])
def test_act_wgrad_many_tiles(T, N, H, dtype):
    say(f"case: act_wgrad many tiles T {T} N {N} H {H} {dtype}")
    g = gen(18)
    dy = randn(g, T, N, dtype=dtype)
    kept = sco().act_pack(randn(g, T, H))
    n = sco().act_unpack(kept, torch.float32).cpu().to(F64)
    d64 = dy.cpu().to(F64)
    ref, mag = (d64.t() @ n).cuda(), (d64.abs().t() @ n.abs()).cuda()
    terms = T * (1 if dtype == torch.bfloat16 else 3) + 64
    within("dW", sco().act_wgrad(dy, kept), ref, ref.abs() * (HALF[dtype] + U) + terms * 2 * U * mag)


@pytest.mark.parametrize("dtype", DT)
def test_xent_many_tiles(dtype):
    T, V, H = 300, 70003, 72
    say(f"case: xent many tiles T {T} V {V} H {H} {dtype}")
    g = gen(19)
    h, W, tgt = _xent_case(g, T, V, H, dtype)
    tgt[5] = -1
    tgt[6] = V - 1
    ref, tol = _xent_ref(h, W, tgt, dtype)
    _xent_check(sco().xent(h, W, tgt), ref, tol)


# ---- the operators together ------------------------------------------------------------------

def test_example_learns():
    """The example's model, trained by its own loop: the loss starts at the uniform distribution's
    and falls."""
    from examples.training_step import Model, train
    losses = train(steps=40)
    assert all(math.isfinite(x) for x in losses)
    assert abs(losses[0] - math.log(512)) < 0.5
    assert sum(losses[-5:]) / 5 < 0.8 * losses[0]


def test_example_gradients_against_differences():
    """The loss falls along the negative gradients by their squared norm, to first order.  The
    checkpoints' rounding (a 127th of a block's largest value) bounds what the gradients that
    read them are off by."""
    from examples.training_step import Model
    g = gen(20)
    m = Model(V=64, H=64, seed=3)
    ids = torch.randint(0, 64, (400,), generator=g, device="cuda")
    tgt = torch.randint(-1, 64, (400,), generator=g, device="cuda")
    _, grads, dgains = m.step(ids, tgt)
    params = m.matrices() + m.gain
    every = grads + dgains
    norm2 = sum((d.double() ** 2).sum() for d in every)
    t = 1e-3 / float(norm2.sqrt())
    losses = []
    for sign in (1, -1):
        for p, d in zip(params, every):
            p.add_(sign * t * d)
        losses.append(float(m.step(ids, tgt)[0]))
        for p, d in zip(params, every):
            p.sub_(sign * t * d)
    slope = (losses[0] - losses[1]) / (2 * t)
    # float32 losses: 2 roundings of about 40 U each over 2 t; checkpoints: half a step of 1/64 of
    # a block's largest power of two, at most 1% of the largest value, twice
    slack = 80 * U * losses[0] / t + 0.04 * float(norm2)
    assert abs(slope - float(norm2)) <= slack
