"""Refusals of the token losses, layer norm and gradient clipping without a GPU: the C entries check
their arguments before any GPU work, the binding checks tensors before it calls them."""
import ctypes
import os

import pytest
import torch

import spectral_correction_optimizer_amd as sco

INVALID, SHAPE = -1, -2
P = ctypes.c_void_p(4096)  # aligned, never read: every call below is refused
ODD = ctypes.c_void_p(4098)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(sco.library_path()):
        pytest.skip("libscopt.so not built")
    return sco.load_library()


def test_token_logp_refusals(lib):
    n = ctypes.c_int64()
    q = lib.sc_token_logp_workspace
    assert q(5, 100, 1000, 64, ctypes.byref(n)) == INVALID
    assert q(1, -1, 1000, 64, ctypes.byref(n)) == SHAPE
    assert q(1, 100, 0, 64, ctypes.byref(n)) == SHAPE
    assert q(1, 100, 1000, 65536, ctypes.byref(n)) == SHAPE
    assert q(1, 100, 1000, 64, None) == INVALID
    assert q(1, 100, 1000, 64, ctypes.byref(n)) == 0 and n.value > 0
    f = lib.sc_token_logp
    assert f(1, ODD, P, P, 100, 1000, 64, P, P, n.value, None) == INVALID
    assert f(1, P, P, P, 100, 1000, 64, None, P, n.value, None) == INVALID
    assert f(1, P, P, P, 100, 1000, 64, P, P, n.value - 1, None) == INVALID
    assert "workspace" in lib.sc_last_error().decode()
    assert f(1, None, None, None, 0, 1000, 64, None, None, 0, None) == 0  # no token: nothing to do


def policy(lib, n, dtype=1, h=P, W=P, tgt=P, old=P, adv=P, ref=P, w=None, T=100, V=1000, H=64, lo=0.2, hi=0.2, kl=0.1,
           limit=0, loss=P, total=P, klm=P, clipped=P, logp=P, dh=P, dW=P, ws=P):
    return lib.sc_policy_loss(dtype, h, W, tgt, old, adv, ref, w, T, V, H, lo, hi, kl, limit, loss, total, klm, clipped,
                              logp, dh, dW, ws, n, None)


def test_policy_refusals(lib):
    n = ctypes.c_int64()
    assert lib.sc_token_loss_workspace(1, 100, 1000, 64, -1, ctypes.byref(n)) == INVALID
    assert lib.sc_token_loss_workspace(1, 100, 1000, 64, 0, None) == INVALID
    assert lib.sc_token_loss_workspace(1, 100, 1000, 64, 0, ctypes.byref(n)) == 0
    n = n.value
    nan, inf = float("nan"), float("inf")
    for bad in (dict(dtype=2), dict(h=ODD), dict(W=None), dict(tgt=None), dict(old=None), dict(adv=ODD), dict(lo=-0.1),
                dict(lo=1.5), dict(lo=nan), dict(hi=-0.1), dict(hi=nan), dict(kl=-1.0), dict(kl=nan), dict(kl=inf),
                dict(ref=None), dict(ref=None, klm=None), dict(ref=None, kl=0.0), dict(limit=-1), dict(loss=None),
                dict(total=None), dict(clipped=None), dict(logp=None), dict(dh=None), dict(dW=None), dict(ws=None),
                dict(w=ODD), dict(ws=ODD)):
        assert policy(lib, n, **bad) == INVALID, bad
    assert policy(lib, n - 1) == INVALID
    for bad in (dict(T=-1), dict(V=1 << 21), dict(H=0)):
        assert policy(lib, 1 << 50, **bad) == SHAPE, bad


def test_preference_refusals(lib):
    n = ctypes.c_int64()
    assert lib.sc_token_loss_workspace(0, 100, 1000, 64, 0, ctypes.byref(n)) == 0

    def call(n=n.value, h=P, starts=P, ref=P, pairs=3, T=100, beta=0.1, margin=0.0, eps=0.0, loss=P, mean=P, rewards=P,
             dW=P):
        return lib.sc_preference_loss(0, h, P, P, starts, ref, pairs, T, 1000, 64, beta, margin, eps, 0, 0, loss, mean,
                                      rewards, P, P, dW, P, n, None)

    nan = float("nan")
    for bad in (dict(h=ODD), dict(starts=None), dict(starts=ODD), dict(ref=ODD), dict(beta=-1.0), dict(beta=nan),
                dict(margin=nan), dict(eps=-0.1), dict(eps=1.1), dict(eps=nan), dict(loss=None), dict(mean=None),
                dict(rewards=None), dict(dW=None), dict(n=n.value - 1)):
        assert call(**bad) == INVALID, bad
    assert call(pairs=-1) == SHAPE and call(pairs=(1 << 20) + 1) == SHAPE


def test_layernorm_refusals(lib):
    f = lib.sc_layernorm
    assert f(3, P, None, P, P, 1e-5, 4, 64, P, P, P, P, P, P, None) == INVALID
    assert f(0, P, None, P, P, 1e-5, 4, 16385, P, P, P, P, P, P, None) == SHAPE
    assert f(0, P, None, P, P, -1.0, 4, 64, P, P, P, P, P, P, None) == INVALID
    assert f(0, P, None, P, P, float("nan"), 4, 64, P, P, P, P, P, P, None) == INVALID
    assert f(0, P, None, None, P, 1e-5, 4, 64, P, P, P, P, P, P, None) == INVALID
    assert f(0, P, ODD, P, P, 1e-5, 4, 64, P, P, P, P, P, P, None) == INVALID
    assert f(0, P, None, P, ODD, 1e-5, 4, 64, P, P, P, P, P, P, None) == INVALID
    assert f(0, P, None, P, P, 1e-5, 4, 64, P, P, None, P, P, P, None) == INVALID
    assert f(0, P, None, P, P, 1e-5, 4, 64, P, P, P, P, P, None, None) == INVALID  # q without e
    n = ctypes.c_int64()
    assert lib.sc_layernorm_grad_workspace(4, 64, None) == INVALID
    assert lib.sc_layernorm_grad_workspace(4, 64, ctypes.byref(n)) == 0
    g, n = lib.sc_layernorm_grad, n.value
    assert g(0, P, P, P, P, P, None, None, None, 4, 64, P, P, P, P, n - 1, None) == INVALID
    assert g(0, P, P, P, P, None, None, None, None, 4, 64, P, P, P, P, n, None) == INVALID  # q without e
    assert g(0, P, P, P, None, None, P, None, None, 4, 64, P, P, P, P, n, None) == INVALID  # h without mean
    assert g(0, P, P, P, P, P, P, P, None, 4, 64, P, P, P, P, n, None) == INVALID  # both
    assert g(0, P, P, P, None, None, None, None, None, 4, 64, P, P, P, P, n, None) == INVALID  # neither
    assert g(0, P, P, P, P, P, None, None, ODD, 4, 64, P, P, P, P, n, None) == INVALID
    assert g(0, P, P, P, P, P, None, None, None, 4, 64, P, None, P, P, n, None) == INVALID


def test_clip_refusals(lib):
    dts, sizes = (ctypes.c_int * 2)(0, 1), (ctypes.c_int64 * 2)(100, 9)
    ptrs = (ctypes.c_void_p * 2)(4096, 8192)
    n = ctypes.c_int64()
    q = lib.sc_grad_sumsq_workspace
    assert q(2, dts, sizes, ctypes.byref(n)) == 0 and n.value == 16
    assert q(0, None, None, ctypes.byref(n)) == 0 and n.value == 0
    assert q(-1, dts, sizes, ctypes.byref(n)) == INVALID
    assert q(2, None, sizes, ctypes.byref(n)) == INVALID
    assert q(2, dts, sizes, None) == INVALID
    assert q(2, (ctypes.c_int * 2)(0, 9), sizes, ctypes.byref(n)) == INVALID
    assert q(2, dts, (ctypes.c_int64 * 2)(100, -1), ctypes.byref(n)) == SHAPE
    assert q(2, dts, (ctypes.c_int64 * 2)(1 << 48, 1 << 48), ctypes.byref(n)) == SHAPE
    f = lib.sc_grad_sumsq
    assert f(2, dts, sizes, ptrs, None, P, 16, None) == INVALID
    assert f(2, dts, sizes, None, P, P, 16, None) == INVALID
    assert f(2, dts, sizes, (ctypes.c_void_p * 2)(4096, None), P, P, 16, None) == INVALID
    assert f(2, dts, sizes, (ctypes.c_void_p * 2)(4098, 4096), P, P, 16, None) == INVALID
    assert f(2, dts, sizes, ptrs, P, P, 15, None) == INVALID
    c = lib.sc_clip_grads
    assert c(2, dts, sizes, ptrs, None, P, 1.0, P, P, None) == INVALID
    assert c(2, dts, sizes, ptrs, ptrs, None, 1.0, P, P, None) == INVALID
    assert c(2, dts, sizes, ptrs, ptrs, P, -1.0, P, P, None) == INVALID
    assert c(2, dts, sizes, ptrs, ptrs, P, float("nan"), P, P, None) == INVALID
    assert c(2, dts, sizes, ptrs, ptrs, P, 1.0, None, P, None) == INVALID


def test_workspace_queries_without_tokens(lib):
    n = ctypes.c_int64()
    for V, H in [(1, 1), (513, 8), (1 << 20, 64)]:
        for dt in (0, 1):
            assert lib.sc_token_logp_workspace(dt, 0, V, H, ctypes.byref(n)) == 0
            assert lib.sc_token_loss_workspace(dt, 0, V, H, 0, ctypes.byref(n)) == 0
    assert lib.sc_layernorm_grad_workspace(0, 64, ctypes.byref(n)) == 0 and n.value == 0


def test_token_logp_holds_no_logits(lib):
    """Its workspace is the rows' statistics, a copy of h and one round of tiles' partial sums: far from T x V."""
    n = ctypes.c_int64()
    assert lib.sc_token_logp_workspace(1, 8192, 131072, 2048, ctypes.byref(n)) == 0
    assert n.value < 8192 * 131072 * 2 // 12


def test_binding_refuses_cpu_tensors_and_shapes():
    x, g, f = torch.zeros(4, 64), torch.zeros(64), torch.zeros(4)
    ids = torch.zeros(4, dtype=torch.int64)
    kept = sco.ActCheckpoint(x.to(torch.int8), torch.zeros(4, 2, dtype=torch.uint8))
    for call in (lambda: sco.token_logp(x, x, ids), lambda: sco.policy_loss(x, x, ids, f, f),
                 lambda: sco.preference_loss(x, x, ids, ids[:3]), lambda: sco.layernorm(x, g),
                 lambda: sco.layernorm_grad(x, g, f, kept=kept), lambda: sco.grad_sumsq([x]),
                 lambda: sco.clip_grads([x], 1.0),
                 # neither the checkpoint nor h and mean; both; h alone
                 lambda: sco.layernorm_grad(x, g, f), lambda: sco.layernorm_grad(x, g, f, kept=kept, h=x, mean=f),
                 lambda: sco.layernorm_grad(x, g, f, h=x), lambda: sco.policy_loss(x, x, ids, f, f, kl=0.1),
                 lambda: sco.token_logp(x.half(), x.half(), ids), lambda: sco.token_logp(g, x, ids),
                 lambda: sco.clip_grads([], 1.0), lambda: sco.grad_sumsq([])):
        with pytest.raises(ValueError):
            call()


def test_clip_norm_refusals(lib):
    dts, sizes = (ctypes.c_int * 2)(0, 1), (ctypes.c_int64 * 2)(100, 9)
    ptrs = (ctypes.c_void_p * 2)(4096, 8192)
    c = lib.sc_clip_norm
    assert c(2, dts, sizes, None, ptrs, 1.0, P, P, P, 16, None) == INVALID
    assert c(2, dts, sizes, ptrs, None, 1.0, P, P, P, 16, None) == INVALID
    assert c(2, dts, sizes, ptrs, (ctypes.c_void_p * 2)(4096, 4097), 1.0, P, P, P, 16, None) == INVALID
    assert c(2, dts, sizes, ptrs, ptrs, -1.0, P, P, P, 16, None) == INVALID
    assert c(2, dts, sizes, ptrs, ptrs, float("nan"), P, P, P, 16, None) == INVALID
    assert c(2, dts, sizes, ptrs, ptrs, 1.0, None, P, P, 16, None) == INVALID
    assert c(2, dts, sizes, ptrs, ptrs, 1.0, P, None, P, 16, None) == INVALID
    assert c(2, dts, sizes, ptrs, ptrs, 1.0, P, P, P, 15, None) == INVALID
    assert c(2, dts, sizes, ptrs, ptrs, 1.0, P, P, None, 16, None) == INVALID
    assert c(2, dts, (ctypes.c_int64 * 2)(100, -1), ptrs, ptrs, 1.0, P, P, P, 16, None) == SHAPE


def test_anchor_read_wait_refuses_no_handle(lib):
    assert lib.sc_anchor_read_wait(None, None) == INVALID
