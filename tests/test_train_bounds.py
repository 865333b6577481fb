"""The root-mean-square bounds of the float32 products, and what they see: a product that leaves out
one of the three bfloat16 planes of an operand is outside (the mistake is planted in a plain product on
the CPU).

A float32 rounding is off by at most U = 2^-24 of the value.  The roundings of a sum are independent,
no partial sum is larger than the sum in the mean over random terms, and a matrix instruction adds 32
terms at once: `segments` products of K terms make segments * K / 32 additions.  16 more (squared: 4 U) are
for the planes that are left out (2^-23 = 2 U of a term at most), the join of splits and the store."""
import math

import pytest
import torch

U = 2.0 ** -24


def rms_bound(segments, K, own=0.0):
    """Bound of the error's norm over the result's; own: the operands' own error in units of U."""
    return U * math.sqrt(segments * math.ceil(K / 32) + 16 + own * own)


def rms(got, ref):
    got, ref = got.double(), ref.double()
    return float((got - ref).norm() / ref.norm())


def two_planes(x):
    """x without its third bfloat16 plane."""
    hi = x.bfloat16().float()
    return hi + (x - hi).bfloat16().float()


# the products of tests/test_gpu_train_accuracy.py: outputs M x N, K terms
@pytest.mark.parametrize("M,N,K,segments,own", [(96, 200, 2, 3, 0), (65, 33, 63, 3, 0), (96, 200, 1999, 3, 0),
                                                (300, 2, 520, 6, 0), (300, 520, 700, 6, 14), (700, 520, 300, 6, 14)])
def test_bound_sees_a_missing_plane(M, N, K, segments, own):
    g = torch.Generator().manual_seed(1)
    a, b = torch.randn(M, K, generator=g), torch.randn(K, N, generator=g)
    ref = a.double() @ b.double()
    bound = rms_bound(segments, K, own)
    assert rms(two_planes(a).double() @ b.double(), ref) > bound
    if segments == 6:  # the other operand has three planes too
        assert rms(a.double() @ two_planes(b).double(), ref) > bound
    # and float32's own sums are inside
    assert rms(a @ b, ref) < bound
