"""The policy update example: its gradients against torch's float64 autograd of
the whole loss, and a few steps that have to lower the distillation loss."""
import numpy as np
import pytest
import torch

from fp8_precision_rollout_gb300 import policy_step as ps
from gpu_helpers import device

pytestmark = pytest.mark.gpu


def test_gradients_are_those_of_the_whole_loss():
    dev = device()
    head = ps.Head(1000, 128, device=dev)
    x, y, adv, ids, u = ps.synthetic_batch(96, 1000, 128, top_k=7, device=dev)
    r = ps.policy_step(head, x, y, adv, ids, u, distill_weight=0.5)
    xd = x.double().requires_grad_()
    wd = head.weight.double().requires_grad_()
    lq = torch.log_softmax(xd @ wd.T, 1)
    kept = y >= 0
    n = kept.sum()
    logp = lq.gather(1, y.clamp(min=0).long()[:, None])[:, 0]
    roll = torch.log_softmax(x.double() @ head.rollout_weight().double().T, 1)
    roll = roll.gather(1, y.clamp(min=0).long()[:, None])[:, 0]
    w = torch.exp(logp.detach() - roll).clamp(max=2.0)
    policy = (torch.where(kept, -w * adv.double() * logp, 0.0)).sum() / n
    p = torch.softmax(u.double(), 1)
    kl = (p * (p.log() - lq.gather(1, ids.long()))).sum(1)
    kl = torch.where(kept, kl, 0.0).sum() / n
    gx, gw = torch.autograd.grad(policy + 0.5 * kl, (xd, wd))
    policy, kl = policy.detach(), kl.detach()
    assert abs(float(r["policy_loss"]) - float(policy)) < 1e-4 * max(1.0, abs(float(policy)))
    assert abs(float(r["distill_loss"]) - float(kl)) < 1e-4 * float(kl)
    # each of the two terms is rounded to BF16 twice (G, result): 1.5 x 2^-8 of its norm,
    # and the two partly cancel in the sum by less than half of it
    for got, want in ((r["grad_hidden"], gx), (r["grad_weight"], gw)):
        assert float((got.double() - want).norm()) <= 2 * 1.5 * 2.0 ** -8 * float(want.norm())
    assert (r["grad_hidden"][~kept] == 0).all()


def test_steps_lower_the_distillation_loss():
    device()
    out = ps.main(["--steps", "4", "--tokens", "256", "--hidden", "256", "--vocab", "4096"])
    kl = [b for _, b in out]
    assert all(np.isfinite(v) for pair in out for v in pair)
    assert kl[-1] < kl[0]
