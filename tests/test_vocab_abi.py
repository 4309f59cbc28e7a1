"""Refusals of the vocabulary operators, on the host before anything is
launched, and their workspace sizes (no GPU needed)."""
import pytest
import torch

import __graft_entry__
from fp8_precision_rollout_gb300 import binding

FAKE = 1 << 20      # aligned, never dereferenced: every call fails its checks first
BIG = 1 << 40
INVALID, ALIGNMENT, SHAPE = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return binding.load()


# name -> (argument names, defaults); the four calls share most of them
_COMMON = dict(hidden=FAKE, ldh=64, weight=FAKE, ldw=64, tokens=4, hidden_dim=64, vocab=100,
               logit_scale=1.0, workspace=FAKE, workspace_bytes=BIG, stream=None)
_CALLS = {
    "token_logprobs": ("hidden ldh weight ldw targets tokens hidden_dim vocab logit_scale logp lse "
                       "workspace workspace_bytes stream"),
    "token_logprobs_backward": ("hidden ldh weight ldw targets lse grad tokens hidden_dim vocab "
                                "logit_scale grad_hidden grad_weight workspace workspace_bytes stream"),
    "distill_topk": ("hidden ldh weight ldw ids logits top_k tokens hidden_dim vocab logit_scale "
                     "loss lse workspace workspace_bytes stream"),
    "distill_topk_backward": ("hidden ldh weight ldw ids logits top_k lse grad tokens hidden_dim "
                              "vocab logit_scale grad_hidden grad_weight workspace workspace_bytes "
                              "stream"),
}


def _call(lib, name, **change):
    a = dict(_COMMON, targets=FAKE, logp=FAKE, lse=FAKE, loss=FAKE, grad=FAKE, grad_hidden=FAKE,
             grad_weight=FAKE, ids=FAKE, logits=FAKE, top_k=5)
    a.update(change)
    return getattr(lib, "fp8rl_" + name)(*[a[k] for k in _CALLS[name].split()])


@pytest.mark.parametrize("name", sorted(_CALLS))
def test_refusals(lib, name):
    bad = [
        (dict(tokens=-1), INVALID), (dict(vocab=-5), INVALID), (dict(vocab=0), SHAPE),
        (dict(vocab=1 << 31), SHAPE), (dict(tokens=1 << 31), SHAPE),
        (dict(hidden_dim=0), SHAPE), (dict(hidden_dim=60), SHAPE),
        (dict(hidden_dim=1 << 21, ldh=1 << 21, ldw=1 << 21), SHAPE),
        (dict(logit_scale=0.0), INVALID), (dict(logit_scale=-1.0), INVALID),
        (dict(logit_scale=float("inf")), INVALID), (dict(logit_scale=float("nan")), INVALID),
        (dict(ldh=56), INVALID), (dict(ldw=0), INVALID), (dict(ldh=68), ALIGNMENT),
        (dict(ldw=68), ALIGNMENT), (dict(hidden=FAKE + 8), ALIGNMENT),
        (dict(weight=FAKE + 2), ALIGNMENT), (dict(lse=FAKE + 2), ALIGNMENT),
        (dict(workspace=FAKE + 16), ALIGNMENT), (dict(workspace_bytes=1000), INVALID),
        (dict(hidden=None), INVALID), (dict(weight=None), INVALID), (dict(lse=None), INVALID),
        (dict(workspace=None), INVALID),
    ]
    if name.startswith("token"):
        bad += [(dict(targets=None), INVALID), (dict(targets=FAKE + 1), ALIGNMENT)]
    else:
        bad += [(dict(ids=None), INVALID), (dict(logits=None), INVALID), (dict(top_k=0), SHAPE),
                (dict(top_k=257), SHAPE), (dict(ids=FAKE + 2), ALIGNMENT),
                (dict(logits=FAKE + 2), ALIGNMENT)]
    if name.endswith("backward"):
        bad += [(dict(grad=None), INVALID), (dict(grad_hidden=None, grad_weight=None), INVALID),
                (dict(grad_hidden=FAKE + 8), ALIGNMENT), (dict(grad_weight=FAKE + 8), ALIGNMENT)]
    for change, want in bad:
        assert _call(lib, name, **change) == want, (change, binding.last_error())
        assert binding.last_error()


def test_workspace_covers_the_need_and_stays_bounded(lib):
    ws = binding.vocab_workspace_bytes
    for bad in ((-1, 64, 100, 0, 0), (4, 60, 100, 0, 0), (4, 64, 0, 0, 0), (4, 64, 100, 257, 0),
                (4, 64, 100, -1, 0)):
        assert ws(*bad) == 0
    assert ws(0, 64, 100) > 0
    # one byte too few is refused, and the message says how many are needed
    need = ws(1000, 512, 5000, 0, False)
    assert _call(lib, "token_logprobs", tokens=1000, hidden_dim=512, ldh=512, ldw=512, vocab=5000,
                 workspace_bytes=need - 1) == INVALID
    assert str(need) in binding.last_error()
    # never the logits: 64 x 20480 tokens over 2^17 words would be 2 x 10^11 of them
    t, h, v = 64 * 20480, 4096, 1 << 17
    assert ws(t, h, v) < 1 << 30
    # backward: packed rows, FP32 sums and one piece of G, a few times the hidden states
    assert ws(t, h, v, 0, True) < 4 * (t * h * 2)
    assert ws(4096, 4096, v, 0, True) < 1 << 30


def test_binding_checks_types_and_shapes_before_the_library():
    cpu = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        binding.token_logprobs(cpu, cpu, torch.zeros(4, dtype=torch.int32))
    with pytest.raises(TypeError):
        binding.distill_topk(cpu, cpu, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2))
