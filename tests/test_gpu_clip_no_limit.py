"""Clipping without a limit: the norm is told, and the gradients stay as they are."""
import math

import pytest
import torch

from tests.test_gpu_train import gen, randn, sco

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("value", [1.0, math.inf, -math.inf, math.nan])
def test_no_limit(value, given):
    m, g = sco(), gen(95)
    grads = [randn(g, 700), randn(g, 33, 5).bfloat16()]
    grads[0][3] = value
    before = [x.clone() for x in grads]
    out = [torch.empty_like(x) for x in grads]
    r = m.clip_grads(grads, math.inf, out=out, sumsq=m.grad_sumsq(grads) if given else None)
    if math.isnan(value):
        assert r.norm.isnan() and r.scale.isnan() and all(x.isnan().all() for x in out)
        return
    assert r.norm.isinf() == math.isinf(value) and r.scale.item() == 1.0
    m.clip_grads(grads, math.inf)
    for x, y, z in zip(before, grads, out):
        assert torch.equal(x, y) and torch.equal(x, z)
    # a limit, however high, and an infinite norm: scale 0
    if math.isinf(value):
        assert m.clip_grads(grads, 3e38, out=out).scale.item() == 0.0
