"""Pins of the oracle's vocabulary operators, against things other than itself:
torch's float64 log_softmax and kl_div with their autograd derivatives, closed
forms (a uniform head; a one-word vocabulary), and central differences."""
import numpy as np
import torch

import oracle


def _head(t, h, v, seed=0):
    g = torch.Generator().manual_seed(seed)
    hid = torch.randn(t, h, generator=g).to(torch.bfloat16)
    w = (torch.randn(v, h, generator=g) * 0.3).to(torch.bfloat16)
    return hid, w, g


def test_logprobs_and_gradients_match_torch_autograd_float64():
    hid, w, g = _head(7, 24, 31)
    y = torch.tensor([0, 30, -1, 5, 5, 17, -100])
    up = torch.randn(7, generator=g, dtype=torch.float64)
    x, ww = hid.double().requires_grad_(), w.double().requires_grad_()
    lq = torch.log_softmax(0.75 * x @ ww.T, 1)
    kept = y >= 0
    logp = torch.where(kept, lq.gather(1, y.clamp(min=0)[:, None])[:, 0], 0.0)
    gx, gw = torch.autograd.grad((up * logp).sum(), (x, ww))
    got, lse = oracle.token_logprobs(hid, w, y.numpy(), 0.75)
    assert np.allclose(got, logp.detach().numpy(), atol=1e-12)
    assert (lse[[2, 6]] == 0).all()
    d, k = oracle.one_hot_targets(y.numpy(), 31)
    dh, dw, _, _ = oracle.head_gradients(hid, w, d, k, up.numpy(), -1.0, 0.75)
    assert np.allclose(dh, gx.numpy(), atol=1e-12) and np.allclose(dw, gw.numpy(), atol=1e-12)


def test_distillation_matches_torch_kl_div_float64():
    hid, w, g = _head(5, 16, 40, seed=1)
    ids = np.array([[3, 9, 0, 39], [5, -1, 6, 7], [-1, -1, -1, -1], [1, 2, 2, 4], [8, 40, 9, 10]])
    u = torch.randn(5, 4, generator=g, dtype=torch.float64).numpy()
    u[1, 2] = -np.inf
    p, lp, there, kept = oracle.teacher_entries(ids, u, 40, 0.5)
    assert (kept == [True, True, False, True, True]).all()
    assert there.sum(axis=1).tolist() == [4, 2, 0, 4, 3]
    assert np.allclose(p.sum(axis=1), kept)
    dense = oracle.dense_teacher(ids, p, there, 40)
    x, ww = hid.double().requires_grad_(), w.double().requires_grad_()
    lq = torch.log_softmax(0.5 * x @ ww.T, 1)
    # cross entropy to the dense distribution plus the entries' own entropy term
    per = -(torch.from_numpy(dense) * lq).sum(1) + torch.from_numpy((p * lp).sum(axis=1))
    per = torch.where(torch.from_numpy(kept), per, 0.0)
    loss, _ = oracle.distill_topk(hid, w, ids, u, 0.5)
    assert np.allclose(loss, per.detach().numpy(), atol=1e-12)
    # without repeated ids it is kl_div of the two distributions
    kl = torch.nn.functional.kl_div(lq[0], torch.from_numpy(dense[0]), reduction="sum")
    assert abs(loss[0] - float(kl)) < 1e-12
    up = torch.randn(5, generator=g, dtype=torch.float64)
    gx, gw = torch.autograd.grad((up * per).sum(), (x, ww))
    dh, dw, _, _ = oracle.head_gradients(hid, w, dense, kept, up.numpy(), 1.0, 0.5)
    assert np.allclose(dh, gx.numpy(), atol=1e-12) and np.allclose(dw, gw.numpy(), atol=1e-12)


def test_closed_forms():
    hid, w, _ = _head(3, 8, 50, seed=2)
    # zero weights: uniform, logp = -log V whatever the target
    logp, lse = oracle.token_logprobs(hid, torch.zeros(50, 8), [4, 0, 49])
    assert np.allclose(logp, -np.log(50)) and np.allclose(lse, np.log(50))
    # a vocabulary of one word is certain
    logp, _ = oracle.token_logprobs(hid, w[:1], [0, 0, 0])
    assert np.allclose(logp, 0.0)
    # a student equal to a teacher that gives every id has no divergence
    z, _, _ = oracle.head_softmax(hid, w)
    ids = np.tile(np.arange(50), (3, 1))
    loss, _ = oracle.distill_topk(hid, w, ids, z)
    assert np.allclose(loss, 0.0, atol=1e-12)


def test_gradient_matches_central_differences():
    hid, w, g = _head(4, 8, 12, seed=3)
    y, up, e = [1, 11, -1, 6], np.array([0.3, -1.2, 5.0, 0.7]), 1e-6
    d, k = oracle.one_hot_targets(y, 12)
    dh, dw, _, _ = oracle.head_gradients(hid, w, d, k, up, -1.0)
    h0, w0 = hid.double().numpy(), w.double().numpy()
    f = lambda a, b: float((up * oracle.token_logprobs(a, b, y)[0]).sum())  # noqa: E731
    for arr, grad, which in ((h0, dh, 0), (w0, dw, 1)):
        for i in [(0, 0), (1, 3), (3, 7), (2, 2)]:
            lo, hi = arr.copy(), arr.copy()
            lo[i] -= e
            hi[i] += e
            num = (f(hi, w0) - f(lo, w0) if which == 0 else f(h0, hi) - f(h0, lo)) / (2 * e)
            assert abs(num - grad[i]) < 1e-8
