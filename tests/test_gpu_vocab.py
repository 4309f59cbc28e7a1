"""GPU parity of token log-probabilities and top-k distillation, forward and
backward, against the float64 oracle.

Tolerances, from the arithmetic.
Forward.  BF16 products are exact in FP32; a sum of H of them in FP32, in any
order and with truncating additions, is off by at most H 2^-23 times the sum of
magnitudes mag_tv.  dz = H 2^-23 max_v mag_tv bounds a row's logits, and moves
its log-sum-exp by no more.  exp2 of an FP32 argument, the sums of positive
terms (at most 128 in sequence, then a tree and at most 32 + 32 more), log and
the last subtraction add at most EVAL = 256 2^-24 (1 + |z| + |lse|).  So
|lse error| <= dz + EVAL, |logp error| <= 2 dz + 2 EVAL; a distillation loss
is a p-weighted mean of such terms, with |log p| in its evaluation error too.
As those are worst cases, the relative 2-norm is held to 1e-5 as well.
Backward.  G's entries are rounded to BF16 (2^-8 of each, half a step) after an
FP32 evaluation that is off by dG = |g| scale q (dz + EVAL); sums over K terms are off by
K 2^-23 of the magnitudes; the result is rounded to BF16 (2^-8).  The 2-norm is
held to 1.5 x 2^-8 (two independent roundings, each at most 2^-8) of the
result's, plus the norm of what EVAL alone does to G: the calls are given an FP32
log-sum-exp, and a token that is nearly certain has a gradient near 0."""
import numpy as np
import pytest
import torch

import fp8_precision_rollout_gb300 as fp8rl
import oracle
from gpu_helpers import Canary, device, np_f32_bits

pytestmark = pytest.mark.gpu


def _head(t, h, v, dev, seed=0, spread=1.0):
    """Hidden states that lean towards their target's row, as a model's do."""
    g = torch.Generator().manual_seed(1000 * seed + t + 7 * h + 13 * v)
    w = (torch.randn(v, h, generator=g) * (spread * h ** -0.5)).to(torch.bfloat16)
    y = torch.randint(0, v, (t,), generator=g)
    row = w[y].float()
    lean = 12 * torch.rand(t, 1, generator=g) * row / row.square().sum(1, keepdim=True).clamp(min=1e-3)
    x = (torch.randn(t, h, generator=g) + lean).to(torch.bfloat16)
    return x, w, y.to(torch.int32), g


def _mask(y, kind):
    y = y.clone()
    t = y.numel()
    if kind == "alternate":
        y[::2] = -1
    elif kind == "all":
        y[:] = -100
    elif kind == "last only":
        y[: t - 1] = -1
    elif kind == "first only":
        y[1:] = -1
    elif kind == "prompt":
        y[: (2 * t) // 3] = -1
    else:
        assert kind == "none"
    return y


def _teacher(t, k, v, y, g):
    """Entries with absent ids, logits of -inf, dense and spread ids, some repeated."""
    ids = (y[:, None].long().clamp(min=0) + torch.randint(1, max(2, v // 7), (t, 1), generator=g)
           * torch.arange(k)) % v
    near = torch.rand(t, generator=g) < 0.3
    ids[near] = (y[near, None].long().clamp(min=0) + torch.arange(k)) % v
    u = -torch.cumsum(torch.rand(t, k, generator=g), 1)
    u[torch.rand(t, k, generator=g) < 0.05] = float("-inf")
    ids[torch.rand(t, k, generator=g) < 0.1] = -3
    ids[y < 0] = -1
    perm = torch.argsort(torch.rand(t, k, generator=g), 1)
    return ids.gather(1, perm).to(torch.int32), u.gather(1, perm)


def _np(t):
    return t.double().cpu().numpy()


def _close32(got, want, tol, what):
    got = _np(got)
    assert np.isfinite(got).all(), what
    assert (np.abs(got - want) <= tol).all(), "%s: worst %g of its tolerance" % (
        what, np.max(np.abs(got - want) / np.maximum(tol, 1e-300)))
    den = np.linalg.norm(want)
    assert np.linalg.norm(got - want) <= 1e-5 * den + 1e-30, "%s: rel %g" % (
        what, np.linalg.norm(got - want) / max(den, 1e-300))


def _close16(got, want, tol, what, evaluation=0.0):
    got = _np(got)
    assert np.isfinite(got).all(), what
    assert (np.abs(got - want) <= tol + 1e-30).all(), "%s: worst %g of its tolerance" % (
        what, np.max(np.abs(got - want) / np.maximum(tol, 1e-300)))
    den = np.linalg.norm(want)
    near = 1.5 * 2.0 ** -8 * den + np.linalg.norm(evaluation) + 1e-30
    assert np.linalg.norm(got - want) <= near, "%s: rel %g" % (
        what, np.linalg.norm(got - want) / max(den, 1e-300))


def _bounds(x, w, scale):
    z, mag, lse = oracle.head_softmax(x, w, scale)
    dz = x.shape[1] * 2.0 ** -23 * mag.max(axis=1)
    ev = 256 * 2.0 ** -24 * (1 + np.abs(z).max(axis=1) + np.abs(lse))
    return dz, ev


def _check_logp(x, w, y, logp, lse, scale, what=""):
    ref, rl = oracle.token_logprobs(x, w, y.numpy(), scale)
    dz, ev = _bounds(x, w, scale)
    _close32(lse, rl, dz + ev, "lse " + what)
    _close32(logp, ref, 2 * dz + 2 * ev, "logp " + what)
    out = (y.numpy() < 0) | (y.numpy() >= w.shape[0])
    assert (_np(logp)[out] == 0).all() and (_np(lse)[out] == 0).all()


def _check_grads(x, w, dist, kept, up, sign, scale, gh, gw, what=""):
    dh, dw, G, q = oracle.head_gradients(x, w, dist, kept, _np(up), sign, scale)
    dz, ev = _bounds(x, w, scale)
    hd, wd = np.abs(oracle._f64(x)) * kept[:, None], np.abs(oracle._f64(w))
    gmag = np.abs(np.where(kept, _np(up), 0.0))[:, None] * scale
    dG = 2.0 ** -8 * np.abs(G) + gmag * (q * (2 * dz + ev)[:, None] + 2.0 ** -22 * (dist + q))
    t, v = G.shape
    E = gmag * (q + dist) * ev[:, None]
    if gh is not None:
        _close16(gh, dh, 2.0 ** -8 * np.abs(dh) + (dG + v * 2.0 ** -23 * np.abs(G)) @ wd,
                 "grad_hidden " + what, E @ wd)
        assert (_np(gh)[~kept] == 0).all()
    if gw is not None:
        _close16(gw, dw, 2.0 ** -8 * np.abs(dw) + (dG + t * 2.0 ** -23 * np.abs(G)).T @ hd,
                 "grad_weight " + what, E.T @ hd)


SIZES = [(1, 8, 1), (1, 64, 2), (2, 72, 63), (1, 4096, 1000), (3, 136, 129), (16, 256, 4099),
         (63, 64, 128), (64, 1000, 257), (65, 128, 256), (127, 72, 255), (128, 512, 2051),
         (129, 2048, 513), (255, 264, 777), (257, 64, 1024), (300, 1032, 3001), (513, 8, 65)]
MASKS = ["none", "alternate", "prompt", "all", "last only", "first only"]


@pytest.mark.parametrize("t,h,v", SIZES)
def test_logprobs_match_the_oracle(t, h, v):
    dev = device()
    for mask in MASKS if t < 200 else MASKS[:3]:
        for scale in (1.0, 0.6) if mask == "none" else (1.0,):
            x, w, y, _ = _head(t, h, v, dev)
            y = _mask(y, mask)
            a, b = Canary(t, torch.float32, dev), Canary(t, torch.float32, dev)
            need = fp8rl.vocab_workspace_bytes(t, h, v)
            ws = Canary(need, torch.uint8, dev, fill=0xFF)           # any contents will do
            logp, lse = fp8rl.token_logprobs(x.to(dev), w.to(dev), y.to(dev), scale, a.view, b.view,
                                             ws.view)
            torch.cuda.synchronize()
            fp8rl.device_status(0)
            a.check(); b.check(); ws.check()
            _check_logp(x, w, y, logp, lse, scale, "%s %s" % (mask, scale))


@pytest.mark.parametrize("t,h,v", SIZES)
def test_logprob_gradients_match_the_oracle(t, h, v):
    dev = device()
    for mask in MASKS if t < 200 else MASKS[:3]:
        scale = 0.6 if mask == "prompt" else 1.0
        x, w, y, g = _head(t, h, v, dev)
        y = _mask(y, mask)
        up = torch.randn(t, generator=g)
        d, kept = oracle.one_hot_targets(y.numpy(), v)
        _, lse = oracle.token_logprobs(x, w, y.numpy(), scale)
        gh, gw = Canary(t * h, torch.bfloat16, dev), Canary(v * h, torch.bfloat16, dev)
        need = fp8rl.vocab_workspace_bytes(t, h, v, 0, True)
        ws = Canary(need, torch.uint8, dev, fill=0xFF)
        fp8rl.token_logprobs_backward(x.to(dev), w.to(dev), y.to(dev),
                                      torch.from_numpy(lse).float().to(dev), up.to(dev), scale,
                                      gh.view.view(t, h), gw.view.view(v, h), workspace=ws.view)
        torch.cuda.synchronize()
        fp8rl.device_status(0)
        gh.check(); gw.check(); ws.check()
        _check_grads(x, w, d, kept, up, -1.0, scale, gh.view.view(t, h), gw.view.view(v, h), mask)


@pytest.mark.parametrize("t,h,v,k", [(1, 64, 1, 1), (1, 256, 1000, 256), (2, 72, 63, 100), (17, 8, 130, 7),
                                     (64, 520, 257, 33), (129, 256, 2051, 64), (300, 64, 777, 20),
                                     (40, 1024, 4099, 8)])
@pytest.mark.parametrize("mask", ["none", "alternate", "all"])
def test_distillation_matches_the_oracle(t, h, v, k, mask):
    dev = device()
    x, w, y, g = _head(t, h, v, dev, seed=3)
    y = _mask(y, mask)
    ids, u = _teacher(t, k, v, y, g)
    scale = 0.5 if mask == "alternate" else 1.0
    args = (x.to(dev), w.to(dev), ids.to(dev), u.to(dev))
    a, b = Canary(t, torch.float32, dev), Canary(t, torch.float32, dev)
    ws = Canary(fp8rl.vocab_workspace_bytes(t, h, v, k), torch.uint8, dev, fill=0xFF)
    loss, lse = fp8rl.distill_topk(*args, scale, a.view, b.view, ws.view)
    torch.cuda.synchronize()
    fp8rl.device_status(0)
    a.check(); b.check(); ws.check()
    ref, rl = oracle.distill_topk(x, w, ids.numpy(), u.numpy(), scale)
    p, lp, there, kept = oracle.teacher_entries(ids.numpy(), u.numpy(), v, scale)
    dz, ev = _bounds(x, w, scale)
    ev = ev + 256 * 2.0 ** -24 * np.abs(lp).max(axis=1)
    _close32(lse, rl, dz + ev, "lse")
    # (a loss near 0 cancels: its own 2-norm is then no measure, so it is joined by the lse's)
    got = _np(loss)
    assert (np.abs(got - ref) <= 2 * dz + 3 * ev).all()
    assert np.linalg.norm(got - ref) <= 1e-5 * (np.linalg.norm(ref) + np.linalg.norm(rl))
    assert (got[~kept] == 0).all()
    up = torch.randn(t, generator=g)
    gh, gw = Canary(t * h, torch.bfloat16, dev), Canary(v * h, torch.bfloat16, dev)
    ws = Canary(fp8rl.vocab_workspace_bytes(t, h, v, k, True), torch.uint8, dev, fill=0xFF)
    fp8rl.distill_topk_backward(*args, torch.from_numpy(rl).float().to(dev), up.to(dev), scale,
                                gh.view.view(t, h), gw.view.view(v, h), workspace=ws.view)
    torch.cuda.synchronize()
    fp8rl.device_status(0)
    gh.check(); gw.check(); ws.check()
    dense = oracle.dense_teacher(ids.numpy(), p, there, v)
    _check_grads(x, w, dense, kept, up, 1.0, scale, gh.view.view(t, h), gw.view.view(v, h))


@pytest.mark.parametrize("t,h,v,k", [(1, 4096, 3001, 5), (2, 4096, 513, 0), (2, 4104, 700, 40),
                                     (2, 1000, 3, 2), (1, 2056, 20000, 0), (8, 4096, 3001, 0), (5, 72, 1001, 9), (8, 256, 129, 256),
                                     (70, 264, 33000, 0), (128, 64, 32768, 12), (130, 128, 16500, 3),
                                     (389, 136, 20011, 0), (600, 64, 50021, 0), (600, 72, 40000, 70),
                                     (1100, 128, 9000, 0), (4500, 64, 3000, 0)])
def test_every_tile_width_and_row_count(t, h, v, k):
    """Shapes by which path they take: a few tokens, one to eighteen row tiles, head
    tiles of other widths than 256 (few rounds), entries in one launch and two."""
    dev = device()
    x, w, y, g = _head(t, h, v, dev, seed=11)
    y[1::7] = -1
    up = torch.randn(t, generator=g)
    xd, wd, yd = x.to(dev), w.to(dev), y.to(dev)
    if k == 0:
        logp, lse = fp8rl.token_logprobs(xd, wd, yd)
        gh, gw = fp8rl.token_logprobs_backward(xd, wd, yd, lse, up.to(dev))
        _check_logp(x, w, y, logp, lse, 1.0)
        d, kept = oracle.one_hot_targets(y.numpy(), v)
        sign = -1.0
    else:
        ids, u = _teacher(t, k, v, y, g)
        loss, lse = fp8rl.distill_topk(xd, wd, ids.to(dev), u.to(dev))
        gh, gw = fp8rl.distill_topk_backward(xd, wd, ids.to(dev), u.to(dev), lse, up.to(dev))
        ref, rl = oracle.distill_topk(x, w, ids.numpy(), u.numpy())
        dz, ev = _bounds(x, w, 1.0)
        p, lp, there, kept = oracle.teacher_entries(ids.numpy(), u.numpy(), v)
        _close32(lse, rl, dz + ev, "lse")
        assert (np.abs(_np(loss) - ref) <= 2 * dz + 3 * (ev + 256 * 2.0 ** -24 * np.abs(lp).max(axis=1))).all()
        d, sign = oracle.dense_teacher(ids.numpy(), p, there, v), 1.0
    torch.cuda.synchronize()
    fp8rl.device_status(0)
    _check_grads(x, w, d, kept, up, sign, 1.0, gh, gw)


def test_pieces_of_tokens_and_of_the_vocabulary():
    """More tokens than one forward piece holds, and a G that takes several
    vocabulary pieces; sampled rows and columns against the oracle."""
    dev = device()
    t, h, v = 20000, 64, 100003
    g = torch.Generator(device=dev).manual_seed(5)
    x = torch.randn(t, h, generator=g, device=dev).to(torch.bfloat16)
    w = (torch.randn(v, h, generator=g, device=dev) * 0.2).to(torch.bfloat16)
    y = torch.randint(0, v, (t,), generator=g, device=dev, dtype=torch.int32)
    y[::5] = -1
    logp, lse = fp8rl.token_logprobs(x, w, y)
    rows = torch.tensor([0, 1, 2, 63, 8191, 8192, 8193, 16383, 16384, 16386, 19998, 19999])
    xs, ys = x.cpu()[rows], y.cpu()[rows]
    _check_logp(xs, w.cpu(), ys, logp.cpu()[rows], lse.cpu()[rows], 1.0)
    up = torch.randn(t, generator=g, device=dev)
    gh, gw = fp8rl.token_logprobs_backward(x, w, y, lse, up)
    torch.cuda.synchronize()
    fp8rl.device_status(0)
    d, kept = oracle.one_hot_targets(ys.numpy(), v)
    _check_grads(xs, w.cpu(), d, kept, up.cpu()[rows], -1.0, 1.0, gh.cpu()[rows], None)
    # columns: G^T of some vocabulary rows, from 64-bit sums on the device
    cols = torch.tensor([0, 1, 4607, 4608, 50000, 99839, 99840, 100002], device=dev)
    z = x.double() @ w[cols].double().T
    kept = y >= 0
    G = (cols[None, :] == y[:, None]).double() - torch.exp(z - lse.double()[:, None])
    G = torch.where(kept[:, None], up.double()[:, None] * G, 0.0)
    want = _np(G.T @ x.double())
    mag = _np(G.abs().T @ x.double().abs())
    # the lse used is the FP32 one on both sides; logits are off by at most H 2^-23 sum |h w|
    dz = h * 2.0 ** -23 * float((x.abs().double() @ w[cols].abs().double().T).max())
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + dz + 256 * 2.0 ** -24 * 32 + t * 2.0 ** -23) * mag
    _close16(gw[cols], want, tol, "grad_weight columns")


def test_few_tokens_over_more_words_than_a_piece_of_g_holds():
    """Two pieces of the vocabulary with several slices of dX each."""
    dev = device()
    t, h, v = 16, 64, 500003
    x, w, y, g = _head(t, h, v, dev, seed=12)
    y[3] = -1
    y[4], y[5] = v - 1, 0
    up = torch.randn(t, generator=g)
    logp, lse = fp8rl.token_logprobs(x.to(dev), w.to(dev), y.to(dev))
    gh, gw = fp8rl.token_logprobs_backward(x.to(dev), w.to(dev), y.to(dev), lse, up.to(dev))
    torch.cuda.synchronize()
    fp8rl.device_status(0)
    _check_logp(x, w, y, logp, lse, 1.0)
    d, kept = oracle.one_hot_targets(y.numpy(), v)
    _check_grads(x, w, d, kept, up, -1.0, 1.0, gh, gw)


@pytest.mark.parametrize("t", [2, 5])
def test_offsets_past_32_bits(t):
    """Weights and their gradient of more than 2^31 elements: targets and sampled
    rows at the far end, against 64-bit products on the device."""
    dev = device()
    h, v = 16384, 140001
    assert h * v > 2 ** 31
    g = torch.Generator(device=dev).manual_seed(t)
    w = torch.empty(v, h, dtype=torch.bfloat16, device=dev)
    for i in range(0, v, 20000):
        w[i:i + 20000] = torch.randn(min(20000, v - i), h, generator=g, device=dev).mul_(h ** -0.5).to(torch.bfloat16)
    x = torch.randn(t, h, generator=g, device=dev).to(torch.bfloat16)
    y = torch.tensor([v - 1, 131072, 5, 140000 - 3, v - 2][:t], dtype=torch.int32, device=dev)
    up = torch.randn(t, generator=g, device=dev)
    logp, lse = fp8rl.token_logprobs(x, w, y)
    gh, gw = fp8rl.token_logprobs_backward(x, w, y, lse, up)
    torch.cuda.synchronize()
    fp8rl.device_status(0)
    z = torch.cat([x.double() @ w[i:i + 20000].double().T for i in range(0, v, 20000)], 1)
    ref = torch.log_softmax(z, 1).gather(1, y.long()[:, None])[:, 0]
    assert float((logp.double() - ref).norm()) <= 1e-5 * float(ref.norm())
    G = -torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
    G.scatter_add_(1, y.long()[:, None], torch.ones(t, 1, dtype=torch.float64, device=dev))
    G *= up.double()[:, None]
    rows = torch.tensor([0, 1, 131071, 131072, 139776, v - 3, v - 2, v - 1], device=dev)
    want = G[:, rows].T @ x.double()
    assert float((gw[rows].double() - want).norm()) <= 1.5 * 2.0 ** -8 * float(want.norm())
    want = sum(G[:, i:i + 20000] @ w[i:i + 20000].double() for i in range(0, v, 20000))
    assert float((gh.double() - want).norm()) <= 1.5 * 2.0 ** -8 * float(want.norm())


def test_gradient_matches_differences_of_the_forward():
    """Central differences of the library's own forward along directions that
    BF16 represents: hidden states and weights are multiples of 2^-6 of at most
    8 bits, steps are +-2^-4."""
    dev = device()
    t, h, v, e = 48, 64, 300, 2.0 ** -4
    g = torch.Generator().manual_seed(9)
    x = torch.randint(-100, 101, (t, h), generator=g) * 2.0 ** -6
    w = torch.randint(-24, 25, (v, h), generator=g) * 2.0 ** -6
    y = torch.randint(0, v, (t,), generator=g, dtype=torch.int32)
    y[::4] = -1
    up = torch.randn(t, generator=g)
    f = lambda a, b: fp8rl.token_logprobs(a.to(torch.bfloat16).to(dev), b.to(torch.bfloat16).to(dev),  # noqa: E731
                                          y.to(dev))
    _, lse = f(x, w)
    gh, gw = fp8rl.token_logprobs_backward(x.to(torch.bfloat16).to(dev), w.to(torch.bfloat16).to(dev),
                                           y.to(dev), lse, up.to(dev))
    kept = (y >= 0).double().numpy()
    for which, shape, grad in (("hidden", (t, h), gh), ("weight", (v, h), gw)):
        d = torch.randint(-1, 2, shape, generator=g).double() * (torch.rand(shape, generator=g) < 0.1)
        for s in (x + e * d if which == "hidden" else w + e * d,):
            assert (s.to(torch.bfloat16).double() == s).all()
        up_d = up.double().numpy() * kept
        if which == "hidden":
            hi, lo = f(x + e * d, w)[0], f(x - e * d, w)[0]
            move = (d @ w.double().T).abs().max(1).values.numpy()
        else:
            hi, lo = f(x, w + e * d)[0], f(x, w - e * d)[0]
            move = (x.double() @ d.T).abs().max(1).values.numpy()
        num = float((up_d * (_np(hi) - _np(lo))).sum() / (2 * e))
        ana = float((_np(grad) * d.numpy()).sum())
        # third derivative of a log-sum-exp along a line whose logits move at
        # most `move` per unit: at most (2 move)^3; forward error 2e-5 each
        # (1e-5 of |logp| <= 10 would be 1e-4); gradients within 2^-7 of magnitudes
        tol = (np.abs(up_d) * ((2 * move) ** 3 * e * e / 6 + 1e-4 / e)).sum() \
            + 2.0 ** -7 * float(np.abs(_np(grad) * d.numpy()).sum()) + 1e-3
        assert abs(num - ana) <= tol, (which, num, ana, tol)
        assert abs(ana) > 4 * 2.0 ** -7 * float(np.abs(_np(grad) * d.numpy()).sum())


def test_left_out_tokens_may_hold_anything():
    dev = device()
    t, h, v = 150, 128, 700
    x, w, y, g = _head(t, h, v, dev, seed=8)
    y = _mask(y, "alternate")
    up = torch.randn(t, generator=g)
    clean = fp8rl.token_logprobs(x.to(dev), w.to(dev), y.to(dev))
    cg = fp8rl.token_logprobs_backward(x.to(dev), w.to(dev), y.to(dev), clean[1], up.to(dev))
    xd, upd, lsed = x.clone(), up.clone(), clean[1].clone()
    xd[0::4], xd[2::4] = float("nan"), float("inf")
    upd[0::2] = float("nan")
    lsed[0::2] = float("nan")
    dirty = fp8rl.token_logprobs(xd.to(dev), w.to(dev), y.to(dev))
    dg = fp8rl.token_logprobs_backward(xd.to(dev), w.to(dev), y.to(dev), lsed, upd.to(dev))
    for a, b in zip(clean + cg, dirty + dg):
        assert torch.equal(a, b)
    # a kept token's NaN stays in its own row of the outputs
    xd = x.clone()
    xd[5, 3] = float("nan")
    logp, lse = fp8rl.token_logprobs(xd.to(dev), w.to(dev), y.to(dev))
    rest = torch.arange(t) != 5
    assert torch.isnan(logp[5]) and torch.isnan(lse[5])
    assert torch.equal(logp.cpu()[rest], clean[0].cpu()[rest])


def test_infinite_logits_and_teacher_nan():
    dev = device()
    t, h, v = 3, 64, 300
    x, w, y, g = _head(t, h, v, dev, seed=4)
    x = x.abs() + 0.5
    w[7] = float("-inf")                       # a word that is switched off
    y[:] = torch.tensor([3, 7, 299])
    logp, lse = fp8rl.token_logprobs(x.to(dev), w.to(dev), y.to(dev))
    w2 = torch.cat([w[:7], w[8:]])
    _, ref = oracle.token_logprobs(x, w2, [0, 0, 0])
    assert np.abs(_np(lse) - ref).max() < 1e-4
    assert torch.isinf(logp[1]) and logp[1] < 0 and torch.isfinite(logp[[0, 2]]).all()
    u = torch.zeros(t, 4)
    u[1, 2] = float("nan")
    ids = torch.tensor([[1, 2, 3, 4]] * t, dtype=torch.int32)
    loss, _ = fp8rl.distill_topk(x.to(dev), w.to(dev), ids.to(dev), u.to(dev))
    assert torch.isnan(loss[1]) and torch.isfinite(loss[[0, 2]]).all()


def test_row_strides_and_single_outputs():
    dev = device()
    t, h, v = 70, 72, 300
    x, w, y, g = _head(t, h, v, dev, seed=6)
    up = torch.randn(t, generator=g).to(dev)
    big = torch.full((t, h + 56), float("nan"), dtype=torch.bfloat16, device=dev)
    big[:, 16:16 + h] = x.to(dev)
    wig = torch.full((v, 2 * h), float("nan"), dtype=torch.bfloat16, device=dev)
    wig[:, :h] = w.to(dev)
    a = fp8rl.token_logprobs(x.to(dev), w.to(dev), y.to(dev))
    b = fp8rl.token_logprobs(big[:, 16:16 + h], wig[:, :h], y.to(dev))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ga = fp8rl.token_logprobs_backward(x.to(dev), w.to(dev), y.to(dev), a[1], up)
    gb = fp8rl.token_logprobs_backward(big[:, 16:16 + h], wig[:, :h], y.to(dev), a[1], up)
    assert torch.equal(ga[0], gb[0]) and torch.equal(ga[1], gb[1])
    only_h = fp8rl.token_logprobs_backward(x.to(dev), w.to(dev), y.to(dev), a[1], up, need_weight=False)
    only_w = fp8rl.token_logprobs_backward(x.to(dev), w.to(dev), y.to(dev), a[1], up, need_hidden=False)
    assert only_h[1] is None and only_w[0] is None
    assert torch.equal(only_h[0], ga[0]) and torch.equal(only_w[1], ga[1])
    with pytest.raises(ValueError):
        fp8rl.token_logprobs(x.to(dev).T, w.to(dev), y.to(dev))
    with pytest.raises(ValueError):
        fp8rl.token_logprobs(x.to(dev), w.to(dev), y.to(dev)[:-1])
    with pytest.raises(TypeError):
        fp8rl.token_logprobs(x.to(dev).half(), w.to(dev), y.to(dev))
    with pytest.raises(TypeError):
        fp8rl.token_logprobs(x.to(dev), w.to(dev), y.long().to(dev))
    with pytest.raises(TypeError):
        fp8rl.token_logprobs(x.numpy, w.to(dev), y.to(dev))
    with pytest.raises(fp8rl.Fp8rlError):
        fp8rl.token_logprobs(x.to(dev)[:, :60].contiguous(), w.to(dev)[:, :60].contiguous(), y.to(dev))


def test_no_tokens():
    dev = device()
    w = torch.randn(33, 64, device=dev).to(torch.bfloat16)
    x = torch.empty(0, 64, dtype=torch.bfloat16, device=dev)
    y = torch.empty(0, dtype=torch.int32, device=dev)
    f = torch.empty(0, dtype=torch.float32, device=dev)
    logp, lse = fp8rl.token_logprobs(x, w, y)
    assert logp.shape == lse.shape == (0,)
    gh, gw = fp8rl.token_logprobs_backward(x, w, y, f, f)
    assert gh.shape == (0, 64) and (gw == 0).all()


def test_bad_ids_are_left_out_and_reported():
    dev = device()
    t, h, v = 10, 64, 100
    x, w, y, g = _head(t, h, v, dev, seed=2)
    y[3], y[8] = v, 2 ** 31 - 1
    fp8rl.device_status(0)
    logp, lse = fp8rl.token_logprobs(x.to(dev), w.to(dev), y.to(dev))
    with pytest.raises(fp8rl.Fp8rlError) as ei:
        fp8rl.device_status(0)
    assert ei.value.status == 1
    _check_logp(x, w, y, logp, lse, 1.0)
    ids = torch.randint(0, v, (t, 6), generator=g, dtype=torch.int32)
    ids[2, 1] = v
    u = torch.randn(t, 6, generator=g)
    loss, _ = fp8rl.distill_topk(x.to(dev), w.to(dev), ids.to(dev), u.to(dev))
    with pytest.raises(fp8rl.Fp8rlError):
        fp8rl.device_status(0)
    ref, _ = oracle.distill_topk(x, w, ids.numpy(), u.numpy())
    assert np.abs(_np(loss) - ref).max() < 1e-4
    fp8rl.device_status(0)


def test_repeats_bit_for_bit_on_another_stream_and_in_a_graph():
    dev = device()
    t, h, v, k = 200, 256, 5000, 9
    x, w, y, g = (a.to(dev) if hasattr(a, "to") else a for a in _head(t, h, v, dev, seed=1))
    y[::3] = -1
    ids, u = _teacher(t, k, v, y.cpu(), g)
    ids, u = ids.to(dev), u.to(dev)
    up = torch.randn(t, generator=g).to(dev)

    def step(stream=None):
        logp, lse = fp8rl.token_logprobs(x, w, y, stream=stream)
        gh, gw = fp8rl.token_logprobs_backward(x, w, y, lse, up, stream=stream)
        loss, l2 = fp8rl.distill_topk(x, w, ids, u, 0.5, stream=stream)
        dh, dw = fp8rl.distill_topk_backward(x, w, ids, u, l2, up, 0.5, stream=stream)
        return logp, lse, gh, gw, loss, l2, dh, dw

    first = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    other = step(side)                        # the current stream stays the default one
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for o in held:
        o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    fp8rl.device_status(0)
    for a, b, c in zip(first, other, held):
        assert torch.equal(a, b) and torch.equal(a, c)
    assert (np_f32_bits(first[0]) == np_f32_bits(other[0])).all()
