"""Refusals of the training-step operators without a GPU: the C entries check their
arguments before any GPU work, the binding checks tensors before it calls them."""
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


def test_embed_refusals(lib):
    f = lib.sc_embed
    assert f(7, P, P, 4, 8, 8, 1.0, P, None) == INVALID
    assert f(0, P, P, -1, 8, 8, 1.0, P, None) == SHAPE
    assert f(0, P, P, 4, 0, 8, 1.0, P, None) == SHAPE
    assert f(0, P, P, 4, 8, 0, 1.0, P, None) == SHAPE
    assert f(0, None, P, 4, 8, 8, 1.0, P, None) == INVALID
    assert f(0, P, None, 4, 8, 8, 1.0, P, None) == INVALID
    assert f(0, ODD, P, 4, 8, 8, 1.0, P, None) == INVALID
    assert f(0, None, None, 0, 8, 8, 1.0, None, None) == 0  # no token: nothing to do


def test_embed_grad_refusals(lib):
    n = ctypes.c_int64()
    assert lib.sc_embed_grad_workspace(4, (1 << 22) + 1, 8, ctypes.byref(n)) == SHAPE
    assert lib.sc_embed_grad_workspace(4, 8, 8, None) == INVALID
    assert lib.sc_embed_grad_workspace(1 << 30, 8, 8, ctypes.byref(n)) == SHAPE  # 32-bit indexes
    assert lib.sc_embed_grad_workspace((1 << 30) - 1, 8, 1, ctypes.byref(n)) == 0
    assert lib.sc_embed_grad_workspace(1000, 5000, 64, ctypes.byref(n)) == 0 and n.value > 0
    f = lib.sc_embed_grad
    assert f(0, P, P, 1000, 5000, 64, 1.0, P, P, n.value - 1, None) == INVALID
    assert "workspace" in lib.sc_last_error().decode()
    assert f(0, P, P, 1000, 5000, 64, 1.0, P, None, n.value, None) == INVALID
    assert f(0, P, P, 1000, 5000, 64, 1.0, None, P, n.value, None) == INVALID
    assert f(3, P, P, 1000, 5000, 64, 1.0, P, P, n.value, None) == INVALID


def test_act_and_norm_refusals(lib):
    assert lib.sc_act_pack(2, P, 4, 8, P, P, None) == INVALID
    assert lib.sc_act_pack(0, P, 4, 0, P, P, None) == SHAPE
    assert lib.sc_act_pack(0, None, 4, 8, P, P, None) == INVALID
    assert lib.sc_act_unpack(0, P, None, 4, 8, P, None) == INVALID
    assert lib.sc_act_unpack(1, P, P, -1, 8, P, None) == SHAPE
    f = lib.sc_rmsnorm
    assert f(0, P, None, P, 1e-5, 4, 16385, P, P, P, P, P, None) == SHAPE
    assert f(0, P, None, P, -1.0, 4, 64, P, P, P, P, P, None) == INVALID
    assert f(0, P, None, P, float("nan"), 4, 64, P, P, P, P, P, None) == INVALID
    assert f(0, P, None, None, 1e-5, 4, 64, P, P, P, P, P, None) == INVALID
    assert f(0, P, None, P, 1e-5, 4, 64, P, P, P, P, None, None) == INVALID  # q without e
    n = ctypes.c_int64()
    assert lib.sc_rmsnorm_grad_workspace(4, 64, ctypes.byref(n)) == 0
    g = lib.sc_rmsnorm_grad
    assert g(0, P, P, P, P, P, None, 4, 64, P, P, P, n.value - 1, None) == INVALID
    assert g(0, P, P, None, P, P, None, 4, 64, P, P, P, n.value, None) == INVALID
    assert g(0, P, P, P, P, P, None, 4, 64, P, None, P, n.value, None) == INVALID


def test_product_refusals(lib):
    n = ctypes.c_int64()
    assert lib.sc_act_wgrad_workspace(0, 100, 0, 64, ctypes.byref(n)) == SHAPE
    assert lib.sc_act_wgrad_workspace(9, 100, 64, 64, ctypes.byref(n)) == INVALID
    assert lib.sc_act_wgrad_workspace(1, 100, 64, 64, ctypes.byref(n)) == 0 and n.value > 0
    assert lib.sc_act_wgrad(1, ODD, P, P, None, 100, 64, 64, P, P, n.value, None) == INVALID
    assert lib.sc_act_wgrad(1, P, P, P, None, 100, 64, 64, P, P, n.value - 1, None) == INVALID
    assert lib.sc_xent_workspace(1, 100, 1 << 21, 64, 0, ctypes.byref(n)) == SHAPE
    assert lib.sc_xent_workspace(1, 100, 1000, 64, -1, ctypes.byref(n)) == INVALID
    assert lib.sc_xent_workspace(1, 100, 1000, 64, 0, ctypes.byref(n)) == 0
    assert lib.sc_xent(1, ODD, P, P, 100, 1000, 64, 0, P, P, P, P, P, n.value, None) == INVALID
    assert lib.sc_xent(1, P, P, None, 100, 1000, 64, 0, P, P, P, P, P, n.value, None) == INVALID
    assert lib.sc_xent(1, P, P, P, 100, 1000, 64, 0, P, None, P, P, P, n.value, None) == INVALID
    assert lib.sc_xent(1, P, P, P, 100, 1000, 64, 0, P, P, P, P, P, n.value - 1, None) == INVALID


def test_xent_limit_bounds_the_workspace(lib):
    """Past the limit only one piece's values are held: the workspace no longer grows with
    T x V, and it holds at least the piece."""
    n = ctypes.c_int64()
    T, H, limit = 4096, 512, 64 << 20
    assert lib.sc_xent_workspace(1, T, 16384, H, limit, ctypes.byref(n)) == 0
    small = n.value
    assert lib.sc_xent_workspace(1, T, 65536, H, limit, ctypes.byref(n)) == 0
    assert small < n.value < 3 * limit
    assert lib.sc_xent_workspace(1, T, 65536, H, 0, ctypes.byref(n)) == 0
    assert n.value > T * 65536 * 2


def test_workspace_queries_without_tokens(lib):
    n = ctypes.c_int64()
    for V, H in [(1, 1), (513, 8), (1 << 21, 64)]:
        assert lib.sc_embed_grad_workspace(0, V, H, ctypes.byref(n)) == 0
        assert lib.sc_rmsnorm_grad_workspace(0, H, ctypes.byref(n)) == 0
        for dt in (0, 1):
            assert lib.sc_act_wgrad_workspace(dt, 0, min(V, 9999), H, ctypes.byref(n)) == 0
            assert lib.sc_xent_workspace(dt, 0, min(V, 9999), H, 1, ctypes.byref(n)) == 0


def test_binding_refuses_cpu_tensors_and_shapes():
    x, g = torch.zeros(4, 64), torch.zeros(64)
    ids = torch.zeros(4, dtype=torch.int64)
    for call in (lambda: sco.embed(x, ids), lambda: sco.embed_grad(x, ids, 8), lambda: sco.act_pack(x),
                 lambda: sco.rmsnorm(x, g), lambda: sco.xent(x, x, ids),
                 lambda: sco.rmsnorm_grad(x, g, torch.zeros(4), sco.ActCheckpoint(x, x))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        sco.embed_grad(x, torch.zeros(5, dtype=torch.int64), 8)
    with pytest.raises(ValueError):
        sco.embed(g, ids)
    with pytest.raises(ValueError):
        sco.xent(x.half(), x.half(), ids)
