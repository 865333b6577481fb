"""Limits of the training-step operators without a GPU: sizes that no launch can take are
refused before any GPU work."""
import ctypes
import os

import pytest

import spectral_correction_optimizer_amd as sco

SHAPE = -2
P = ctypes.c_void_p(4096)  # aligned, never read: every call below is refused


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(sco.library_path()):
        pytest.skip("libscopt.so not built")
    return sco.load_library()


def test_embed_grad_launch_limit(lib):
    """A launch holds fewer than 2^32 threads: 2^26 wavefronts of stretches and table rows."""
    n = ctypes.c_int64()
    big = 1 << 40
    # 2^19 eights of rows, 128 slabs of columns: one slab more than fits
    for T, V, H in [(0, 1 << 22, 128 * 512), (1, 1 << 22, 1 << 24), ((1 << 30) - 1, 8, 2 * 512)]:
        assert lib.sc_embed_grad_workspace(T, V, H, ctypes.byref(n)) == SHAPE, (T, V, H)
        assert lib.sc_embed_grad(1, P, P, T, V, H, 1.0, P, P, big, None) == SHAPE, (T, V, H)
    for T, V, H in [(0, 1 << 22, 127 * 512), ((1 << 30) - 1, 8, 512), (1 << 29, 8, 513)]:
        assert lib.sc_embed_grad_workspace(T, V, H, ctypes.byref(n)) == 0, (T, V, H)
