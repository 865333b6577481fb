"""What the binding of the operators for adapting a model says where it refuses a call: each by the check that the
call is made for.  The checks of tensors come behind the one of their device, so most need a GPU."""
import pytest
import torch

import spectral_correction_optimizer_amd as sco


def refused(call, match):
    with pytest.raises(ValueError, match=match):
        call()


def test_without_a_gpu():
    x, g, f = torch.zeros(4, 64), torch.zeros(64), torch.zeros(4)
    ids = torch.zeros(4, dtype=torch.int64)
    kept = sco.ActCheckpoint(x.to(torch.int8), torch.zeros(4, 2, dtype=torch.uint8))
    for call in (lambda: sco.token_logp(x, x, ids), lambda: sco.policy_loss(x, x, ids, f, f),
                 lambda: sco.preference_loss(x, x, ids, ids[:3]), lambda: sco.layernorm(x, g),
                 lambda: sco.layernorm_grad(x, g, f, kept=kept), lambda: sco.grad_sumsq([x]),
                 lambda: sco.clip_grads([x], 1.0)):
        refused(call, "must be on a GPU, got cpu")
    for args in (dict(), dict(kept=kept, h=x, mean=f), dict(h=x), dict(mean=f), dict(kept=kept, mean=f)):
        refused(lambda: sco.layernorm_grad(x, g, f, **args), "either kept or h and mean")
    refused(lambda: sco.token_logp(x.half(), x.half(), ids), "float32 or bfloat16, got torch.float16")
    refused(lambda: sco.token_logp(g, x, ids), "h must be a matrix")
    refused(lambda: sco.policy_loss(x, g, ids, f, f), "W must be a matrix")
    refused(lambda: sco.layernorm(g, g), "x must be a matrix")
    refused(lambda: sco.layernorm_grad(g, g, f, kept=kept), "dy must be a matrix")
    for call in (sco.grad_sumsq, lambda grads: sco.clip_grads(grads, 1.0)):
        refused(lambda: call([]), "no tensors")
        refused(lambda: call([3, x]), "entry 0 is a int, not a tensor")
        refused(lambda: call([None]), "entry 0 is a NoneType")


@pytest.mark.gpu
def test_on_a_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    x, g, f = (torch.zeros(*s, device="cuda") for s in ((4, 64), (64,), (4,)))
    ids, starts = torch.zeros(4, dtype=torch.int64, device="cuda"), torch.tensor([0, 2, 4], device="cuda")
    refused(lambda: sco.policy_loss(x, x, ids, f, f, kl=0.1), "kl needs ref_logp")
    wrong = {"h": dict(h=x.t().contiguous().t()), "W": dict(W=x.bfloat16()), "targets": dict(targets=ids.int()),
             "old_logp": dict(old_logp=f.double()), "advantages": dict(advantages=f[:3]), "ref_logp": dict(ref_logp=f.cpu()),
             "weights": dict(weights=f[:, None])}
    for name, other in wrong.items():
        args = dict(h=x, W=x, targets=ids, old_logp=f, advantages=f) | other
        refused(lambda: sco.policy_loss(**args), f"policy_loss: {name} must be a contiguous")
        if name in ("h", "W", "targets", "ref_logp"):
            args = dict(h=x, W=x, targets=ids, starts=starts) | other
            refused(lambda: sco.preference_loss(**args), f"preference_loss: {name} must be a contiguous")
        if name in ("h", "W", "targets"):
            args = dict(h=x, W=x, targets=ids) | other
            refused(lambda: sco.token_logp(**args), f"token_logp: {name} must be a contiguous")
    refused(lambda: sco.token_logp(x, x[:, :60].contiguous(), ids), "W must be a contiguous .* shape .4, 64.")
    for s in (starts[:2], starts.int(), starts[:0], starts.cpu(), starts[:, None]):
        refused(lambda: sco.preference_loss(x, x, ids, s), "starts must be a contiguous torch.int64")
    refused(lambda: sco.layernorm(x, g[:60]), "gain must be a contiguous")
    refused(lambda: sco.layernorm(x, g.bfloat16()), "gain must be a contiguous")
    refused(lambda: sco.layernorm(x, g, bias=x), "bias must be a contiguous")
    refused(lambda: sco.layernorm(x, g, residual=x[:3]), "residual must be a contiguous")
    kept = sco.act_pack(x)
    refused(lambda: sco.layernorm_grad(x, g, f[:2], kept=kept), "rstd must be a contiguous")
    refused(lambda: sco.layernorm_grad(x, g, f, h=x, mean=f.double()), "mean must be a contiguous")
    refused(lambda: sco.layernorm_grad(x, g, f, h=x.bfloat16(), mean=f), "layernorm_grad: h must be a contiguous")
    refused(lambda: sco.layernorm_grad(x, g, f, kept=kept, dh=x[:3]), "dh must be a contiguous")
    refused(lambda: sco.layernorm_grad(x, g, f, kept=sco.ActCheckpoint(kept.q, kept.e[:, :1])), "e must be a contiguous")
    refused(lambda: sco.layernorm_grad(x, g, f, kept=sco.ActCheckpoint(kept.q.float(), kept.e)), "q must be a contiguous")
    refused(lambda: sco.clip_grads([x, 3], 1.0), "entry 1 is a int, not a tensor")
    refused(lambda: sco.clip_grads([x, x.half()], 1.0), "gradient 1 must be a contiguous")
    refused(lambda: sco.clip_grads([x], 1.0, out=[3]), "entry 0 is a int, not a tensor")
    refused(lambda: sco.clip_grads([x], 1.0, out=[x.bfloat16()]), "output 0 must be a contiguous torch.float32")
    refused(lambda: sco.clip_grads([x], 1.0, out=[]), "0 outputs for 1 gradients|no tensors")
    refused(lambda: sco.clip_grads([x], 1.0, sumsq=f[0]), "sumsq must be a contiguous torch.float64")
