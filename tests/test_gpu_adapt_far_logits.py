"""Logits hundreds apart, kept relative to their rows' references: entries far below the target's, down to the smallest
numbers that bfloat16 holds, and targets far below the largest logits."""
import math

import pytest
import torch

from tests.gpu_harness import say
from tests.test_gpu_adapt import Tokens, _policy_inputs, _policy_ref
from tests.test_gpu_train import _xent_case, gen, sco, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# (scale of the states, share of them that it is for, targets as drawn or the row's largest logit's)
@pytest.mark.parametrize("scale,every,largest", [(1e3, 1, False), (100.0, 1, True), (30.0, 2, True), (300.0, 3, False)])
def test_policy_of_far_logits(scale, every, largest):
    say(f"case: policy far logits scale {scale} every {every} largest {largest}")
    g = gen(5)
    T, V, H = 700, 24100, 72
    h, W, tgt = _xent_case(g, T, V, H, torch.bfloat16)
    h[::every] = (h[::every].float() * scale).bfloat16()
    if largest:
        tgt = (h.float() @ W.float().t()).argmax(1)
    ref = Tokens(h, W, tgt, torch.bfloat16)
    old, adv, refl, _ = _policy_inputs(g, ref, (0.2, 0.2))
    out = sco().policy_loss(h, W, tgt, old.cuda(), adv.cuda(), ref_logp=refl.cuda(), kl=0.02)
    loss, dloss, _, _, _, _, c, dc, _ = _policy_ref(ref, old, adv, refl, None, (0.2, 0.2), 0.02)
    within("logp", out.logp.cpu(), ref.logp, ref.dlogp)
    within("loss", out.loss.cpu(), loss, dloss)
    dh, dW, tdh, tdW = ref.gradients(c, dc)
    within("dh", out.dh.cpu(), dh, tdh)
    within("dW", out.dW.cpu(), dW, tdW)
    # the same from pieces, which are relative to nothing: as many entries that are not zero, but for the last ones
    pieces = sco().policy_loss(h, W, tgt, old.cuda(), adv.cuda(), ref_logp=refl.cuda(), kl=0.02, limit=1)
    a, b = (int(torch.count_nonzero(x.dW)) for x in (out, pieces))
    say(f"  entries of dW that are not zero: {a}, {b} from pieces")
    assert a >= 0.99 * b
