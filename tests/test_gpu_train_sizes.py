"""GPU tests of the training-step operators at sizes that their other tests do not reach: the
launch limits of the embedding gradient, and the 256 x 256 tile of the products (the sizes of the other
tests take the 64 x 128 and 128 x 128 tiles), with every way of storing its sums.  The library's
own choice of tile is asked for, so that a size that comes to take another tile fails here."""
import ctypes

import pytest
import torch

from tests.gpu_harness import say
from tests.test_train_bounds import rms, rms_bound

pytestmark = pytest.mark.gpu

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


class Plan(ctypes.Structure):
    """TpPlan of csrc/train.hpp."""
    _fields_ = [(n, ctypes.c_int) for n in ("shape", "bm", "bn", "tiles_m", "tiles_n", "splits")] + \
               [("part_bytes", ctypes.c_int64)]


def plan(M, N, K, nseg, may_split):
    """scopt::tp_plan: the tile and split of an M x N product of nseg segments of K terms."""
    f = sco().load_library()["_ZN5scopt7tp_planEiiiib"]
    f.restype, f.argtypes = Plan, [ctypes.c_int] * 4 + [ctypes.c_bool]
    return f(M, N, K, nseg, may_split)


def large(M, N, K, nseg, split=None):
    """The product takes the 256 x 256 tile, split or not as asked (None: it cannot be)."""
    p = plan(M, N, K, nseg, split is not None)
    assert (p.bm, p.bn) == (256, 256) and (p.splits > 1) == bool(split), (M, N, K, p.bm, p.bn, p.splits)
    return p.tiles_m * p.tiles_n * p.splits


CUS = 256  # workgroups of the 256 x 256 tile that run at once


def test_embed_grad_more_crossings_than_a_launch_holds():
    """Over 2^24 stretches of sorted tokens, and every table row crosses thousands of them: more
    crossings than workgroups of 256 threads fit in one launch.  Small integers: every sum is exact."""
    T, V = (1 << 29) + 12345, 4099
    say(f"case: embed_grad T {T} V {V} H 1")
    dy = torch.randint(-8, 8, (T, 1), generator=gen(1), device="cuda", dtype=torch.int8).float()
    ids = torch.arange(T, device="cuda") % V
    dW = sco().embed_grad(dy, ids, V)
    n = T // V
    ref = dy[:n * V].view(n, V).sum(0, dtype=F64)
    ref[:T - n * V] += dy[n * V:, 0]
    assert torch.equal(dW[:, 0].to(F64), ref)


# ends cut in every direction; stored whole and in splits; the first of each: more tiles than workgroups
@pytest.mark.parametrize("dtype,T,N,H,split", [
    (torch.bfloat16, 1030, 8190, 8180, False), (torch.bfloat16, 8190, 2000, 1032, True),
    (torch.float32, 500, 8190, 8180, False), (torch.float32, 3001, 2000, 1031, True)])
def test_act_wgrad_large_tile(dtype, T, N, H, split):
    from tests.test_gpu_train import HALF, U, randn, within
    say(f"case: act_wgrad large tile T {T} N {N} H {H} {dtype}")
    work = large(N, H, T, 1 if dtype == torch.bfloat16 else 3, split)
    assert split or work > 2 * CUS
    g = gen(2)
    dy, gain = randn(g, T, N, dtype=dtype), randn(g, H, dtype=dtype)
    kept = sco().act_pack(randn(g, T, H))
    n = sco().act_unpack(kept, torch.float32).to(F64)
    d64, gn = dy.to(F64), gain.to(F64)
    # (a transposed left operand is copied: plain 64-bit products of contiguous matrices)
    dt = d64.t().contiguous()
    ref, mag = dt @ n, dt.abs() @ n.abs()
    terms = T * (1 if dtype == torch.bfloat16 else 3) + 64
    dW = sco().act_wgrad(dy, kept, gain=gain)
    within("dW", dW, ref * gn, (ref * gn).abs() * (HALF[dtype] + U) + terms * 2 * U * mag * gn.abs())
    if dtype == torch.float32:
        assert rms(dW, ref * gn) <= rms_bound(3, T)
    assert torch.equal(dW, sco().act_wgrad(dy, kept, gain=gain))


# the logits product with the exponentials (bfloat16) or the logits (float32) kept, and the gradient
# products, split or not; in bfloat16 operands used in place (H % 8 = 0) and copied
@pytest.mark.parametrize("dtype,T,V,H,dh_split,dw_split", [
    (torch.bfloat16, 1999, 16301, 520, True, False), (torch.bfloat16, 1999, 16301, 519, True, False),
    (torch.bfloat16, 4001, 3001, 4001, False, False),
    (torch.float32, 1020, 16301, 264, True, True), (torch.float32, 700, 65500, 261, True, False)])
def test_xent_large_tile(dtype, T, V, H, dh_split, dw_split):
    say(f"case: xent large tile T {T} V {V} H {H} {dtype}")
    nseg = 1 if dtype == torch.bfloat16 else 6
    large(T, V, H, nseg)
    large(T, H, V, nseg, dh_split)
    large(V, H, T, nseg, dw_split)
    _xent(dtype, T, V, H, 0)


# in pieces: nothing kept by the logits product, and the gradients of the recomputed logits
@pytest.mark.parametrize("dtype,T,V,H,piece", [(torch.bfloat16, 1999, 16301, 520, 8192),
                                               (torch.float32, 1020, 32701, 264, 16384)])
def test_xent_large_tile_in_pieces(dtype, T, V, H, piece):
    say(f"case: xent large tile in pieces T {T} V {V} H {H} {dtype}")
    bf16 = dtype == torch.bfloat16
    large(T, piece, H, 1 if bf16 else 6)
    large(T, V % piece, H, 1 if bf16 else 6)
    _xent(dtype, T, V, H, piece * T * (2 if bf16 else 6))


def _xent(dtype, T, V, H, limit):
    from tests.test_gpu_train import _xent_case, _xent_check, _xent_ref
    h, W, tgt = _xent_case(gen(3), T, V, H, dtype)
    tgt[1], tgt[2], tgt[3] = -1, V, V - 1
    out = sco().xent(h, W, tgt, limit=limit)
    ref, tol = _xent_ref(h, W, tgt, dtype)
    _xent_check(out, ref, tol)
    for a, b in zip(out, sco().xent(h, W, tgt, limit=limit)):
        assert torch.equal(a, b)
