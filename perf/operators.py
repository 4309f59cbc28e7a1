"""The vocabulary operators, case by case: their plain forms in torch, and the library's calls.

Two operators over a language-model head (hidden states [T, H] and vocabulary weights [V, H], BF16), each
forward and backward, neither of which keeps the [T, V] logits:

  logp     log-probability of each token's target under softmax(logit_scale * hidden @ weight^T), and the
           log-sum-exp it was normalised with; a token whose target is negative is left out (0, 0).
  distill  cross entropy to a teacher's top entries, as a KL divergence: the teacher's given logits are
           softmax-ed over the entries present (id >= 0, logit not -inf), the student over the whole
           vocabulary; a token without entries is left out (0, 0).

`own` selects what run() does: False, the plain form (32-bit torch operations, rounded once at the end);
True, the calls a user makes of fp8_precision_rollout_gb300.
"""
import math

import torch

own = False

#: work of the largest listed case, in multiply-adds; a drawn one stays below it
MOST = 3 * 4096 * 4096 * 65536
PRODUCTS = {"logp": 1, "logp_grad": 3, "distill": 1, "distill_grad": 3}


def _case(name, op, tokens, hidden, vocab, masked=0.0, k=0, scale=1.0):
    return {"name": name, "op": op, "tokens": tokens, "hidden": hidden, "vocab": vocab, "masked": masked, "k": k, "scale": scale}


def listed():
    return [
        # a tiny head, as in a draft model or a test: nothing but launches
        _case("logp tiny", "logp", 4, 256, 2048),
        # the log-probability of the token one sequence has just sampled, at a temperature
        _case("logp one token", "logp", 1, 4096, 131072, scale=1.25),
        # a decode batch's sampled tokens
        _case("logp decode batch", "logp", 64, 2048, 65536),
        # one odd-sized response behind a prompt that is left out, odd vocabulary
        _case("logp ragged response", "logp", 1021, 2048, 50021, masked=0.4),
        # a policy-update micro-batch: logp_train of every token
        _case("logp training batch", "logp", 4096, 4096, 131072),
        # the gradient for one short response
        _case("logp grad short", "logp_grad", 129, 2048, 32768),
        # the gradient of an odd batch, half of it prompt tokens, at a temperature
        _case("logp grad ragged", "logp_grad", 777, 1032, 20011, masked=0.5, scale=1.25),
        # a policy-update micro-batch's gradient, a quarter of it prompt tokens
        _case("logp grad training batch", "logp_grad", 4096, 4096, 65536, masked=0.25),
        # distillation of a few tokens from eight teacher entries each
        _case("distill few", "distill", 16, 2048, 32768, k=8),
        # a distillation micro-batch, 64 teacher entries a token
        _case("distill batch", "distill", 2048, 4096, 65536, masked=0.1, k=64),
        # a short odd batch's distillation gradient, softened
        _case("distill grad short", "distill_grad", 41, 1024, 16385, masked=0.2, k=20, scale=0.5),
        # the micro-batch's gradient
        _case("distill grad batch", "distill_grad", 2048, 4096, 65536, masked=0.1, k=64),
    ]


def draw(rng):
    op = rng.choice(["logp", "logp_grad", "distill", "distill_grad"])
    hidden = 8 * round(math.exp(rng.uniform(math.log(32), math.log(512))))
    vocab = round(math.exp(rng.uniform(math.log(1000), math.log(131072))))
    tokens = round(math.exp(rng.uniform(0.0, math.log(4096))))
    tokens = max(1, min(tokens, MOST // (PRODUCTS[op] * hidden * vocab)))
    c = _case("", op, tokens, hidden, vocab, masked=rng.choice([0.0, 0.0, 0.1, 0.5]),
              k=rng.randint(1, 100) if op.startswith("distill") else 0, scale=rng.choice([1.0, 1.0, 0.5, 1.25]))
    del c["name"]
    return c


def _left_out(case):
    return int(case["masked"] * case["tokens"])


def prepare(case, seed):
    t, h, v, k = case["tokens"], case["hidden"], case["vocab"], case["k"]
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=dev)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    # weights ~N(0, 1/sqrt(H)), so that unit hidden states give logits ~N(0, 1); the hidden states lean towards
    # their target's row by 0 to 16, as a trained model's do: log-probabilities from near 0 to about -log V - 2
    weight = (normal(v, h) * h ** -0.5).to(torch.bfloat16)
    target = (uniform(t) ** 3 * v).long().clamp_(max=v - 1)          # frequent tokens have low ids
    row = weight[target].float()
    hidden = (normal(t, h) + 16 * uniform(t, 1) * row / row.square().sum(1, keepdim=True)).to(torch.bfloat16)
    out = torch.argsort(uniform(t))[: _left_out(case)]               # which tokens are left out
    s = {"op": case["op"], "scale": case["scale"], "hidden": hidden, "weight": weight}
    if k == 0:
        s["targets"] = target.to(torch.int32)
        s["targets"][out] = -1
    else:
        k_in = min(k, v)
        # each token's entries are distinct: an arithmetic progression around the ids, dense for some tokens
        span = 1 + (uniform(t, 1) ** 3 * (v // k_in - 1)).long()
        ids = (target[:, None] + span * torch.arange(k, device=dev)) % v
        ids = torch.where(torch.arange(k, device=dev) < k_in, ids, -1)
        few = 1 + (uniform(t, 1) * k).long()                         # one token in eight has fewer entries
        ids = torch.where((uniform(t, 1) < 0.125) & (torch.arange(k, device=dev) >= few), -1, ids)
        ids[out] = -1
        s["teacher_ids"] = ids.to(torch.int32)
        # log-probabilities, falling off as a trained teacher's do
        s["teacher_logits"] = -torch.cumsum(-torch.log(uniform(t, k).clamp_(min=1e-6)) * 0.3, 1)
    if case["op"].endswith("grad"):
        # advantages times importance weights, over the number of tokens; the log-sum-exp the forward pass kept
        s["grad"] = normal(t) / max(1, t - _left_out(case))
        # (in pieces of tokens, so that preparing costs no memory that the passes do not)
        s["lse"] = torch.cat([torch.logsumexp(x.float() @ weight.float().T * case["scale"], 1) for x in hidden.split(2048)])
    return s


# ------------------------------------------------------------------ the library's calls --

def _run_own(s):
    import fp8_precision_rollout_gb300 as fp8rl

    op = s["op"]
    if op == "logp":
        logp, lse = fp8rl.token_logprobs(s["hidden"], s["weight"], s["targets"], logit_scale=s["scale"])
        return {"logp": logp, "lse": lse}
    if op == "distill":
        loss, lse = fp8rl.distill_topk(s["hidden"], s["weight"], s["teacher_ids"], s["teacher_logits"], logit_scale=s["scale"])
        return {"loss": loss, "lse": lse}
    if op == "logp_grad":
        gh, gw = fp8rl.token_logprobs_backward(s["hidden"], s["weight"], s["targets"], s["lse"], s["grad"], logit_scale=s["scale"])
    else:
        gh, gw = fp8rl.distill_topk_backward(s["hidden"], s["weight"], s["teacher_ids"], s["teacher_logits"], s["lse"], s["grad"],
                                             logit_scale=s["scale"])
    return {"grad_hidden": gh, "grad_weight": gw}


# ------------------------------------------------------------------------- plain forms --

def _teacher(s):
    """(present entries, their ids, the teacher's probabilities over them, tokens with any)."""
    ids, u = s["teacher_ids"].long(), s["teacher_logits"] * s["scale"]
    there = (ids >= 0) & (u != -math.inf)
    some = there.any(1)
    u = torch.where(there, u, -math.inf)
    e = torch.exp(u - torch.where(some, u.amax(1), 0.0)[:, None])
    return there, ids.clamp(min=0), e / torch.where(some, e.sum(1), 1.0)[:, None], some


def _run_plain(s):
    op = s["op"]
    if s["op"].startswith("logp"):
        some, target = s["targets"] >= 0, s["targets"].long().clamp(min=0)
    else:
        there, ids, p, some = _teacher(s)
    x = torch.where(some[:, None], s["hidden"].float(), 0.0)
    w = s["weight"].float()
    z = (x @ w.T) * s["scale"]
    if op.endswith("grad"):
        d = torch.exp(z - s["lse"][:, None])                     # the softmax
        if op == "logp_grad":
            d.neg_()
            d.scatter_add_(1, target[:, None], torch.ones_like(s["lse"])[:, None])
        else:
            d.scatter_add_(1, ids, torch.where(there, -p, 0.0))
        d *= torch.where(some, s["grad"] * s["scale"], 0.0)[:, None]
        return {"grad_hidden": (d @ w).to(torch.bfloat16), "grad_weight": (d.T @ x).to(torch.bfloat16)}
    top = z.amax(1)
    lse = top + torch.log(torch.exp(z - top[:, None]).sum(1))
    if op == "logp":
        y = z.gather(1, target[:, None])[:, 0] - lse
        return {"logp": torch.where(some, y, 0.0), "lse": torch.where(some, lse, 0.0)}
    log_q = z.gather(1, ids) - lse[:, None]
    term = torch.where(there & (p != 0), p * (torch.log(p) - log_q), 0.0)
    return {"loss": torch.where(some, term.sum(1), 0.0), "lse": torch.where(some, lse, 0.0)}


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    t, h, v, k = case["tokens"], case["hidden"], case["vocab"], case["k"]
    n = t - _left_out(case)                                      # tokens that are not left out
    grad = case["op"].endswith("grad")
    small = 8 * t * k + (4 * t if k == 0 else 0) + 8 * t         # targets or teacher, two vectors in or out
    both = 2 if grad else 1                                      # the gradients have their inputs' shapes
    return {"bytes": 2 * (n * h + v * h) + (both - 1) * 2 * (t * h + v * h) + small,
            "flops": 2 * PRODUCTS[case["op"]] * n * h * v}


def exact(case, seed):
    """The definition in 64 bits, by torch's own log-softmax and, for the gradients, its derivatives."""
    s = prepare(case, seed)
    op, t = s["op"], case["tokens"]
    if op.startswith("logp"):
        kept = (s["targets"] >= 0).nonzero()[:, 0]
    else:
        kept = (s["teacher_ids"] >= 0).any(1).nonzero()[:, 0]
    grad = op.endswith("grad")
    x = s["hidden"][kept].double().requires_grad_(grad)
    w = s["weight"].double().requires_grad_(grad)
    z = torch.nn.functional.linear(x, w) * s["scale"]
    lse = torch.logsumexp(z.detach(), 1)
    log_q = torch.log_softmax(z, 1)
    if op.startswith("logp"):
        y = log_q.gather(1, s["targets"][kept].long()[:, None])[:, 0]
    else:
        ids = s["teacher_ids"][kept].long()
        log_p = torch.log_softmax((s["teacher_logits"][kept].double() * s["scale"]).masked_fill(ids < 0, -math.inf), 1)
        inner = log_p.exp() * (log_p.masked_fill(ids < 0, 0.0) - log_q.gather(1, ids.clamp(min=0)))
        y = inner.masked_fill(ids < 0, 0.0).sum(1)
    full = torch.zeros(t, dtype=torch.float64, device=x.device)
    if not grad:
        return {"logp" if op == "logp" else "loss": full.index_copy(0, kept, y), "lse": full.index_copy(0, kept, lse)}
    del z, log_q
    gx, gw = torch.autograd.grad(y, (x, w), s["grad"][kept].double())
    return {"grad_hidden": torch.zeros(t, case["hidden"], dtype=torch.float64, device=x.device).index_copy(0, kept, gx),
            "grad_weight": gw}
