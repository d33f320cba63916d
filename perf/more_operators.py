"""Cases of the operators over rows of vocabulary logits: log probabilities of given tokens with
entropy and the likeliest alternatives, and distillation from a teacher's top entries with its
gradient.

Next to draft verification a serving step answers with log probabilities, and a draft model is
trained on what the target recorded while it served: the alternatives that ``token_logprobs`` returns
are the teacher entries that ``distill_topk`` takes.

  logprobs      y = s x:  y_token - lse(y), entropy of softmax(y), the k largest entries
  distill       KL(teacher || student) of each row over the teacher's entries, and what its
                gradient needs again
  distill_bwd   the gradient in the logits for a gradient of the losses
  distill_grad  loss and gradient in one call, for losses that are summed with given weights

With q = softmax(s x) the student's probabilities, teacher entries (id_i, v_i), p_i = softmax(v) and
M = 1 the loss is sum_i p_i (log p_i - log q[id_i]) and its gradient in x is s (M q - sum_i p_i
[id_i]).  With ``tail`` v are log probabilities, p_i = exp(v_i), and what they leave, r = max(0, 1 -
sum p), is one more outcome: all tokens outside the entries, of mass q_r.  The loss then has r (log r
- log q_r) more, M = sum p + r, and the gradient -s r q / q_r on the tokens outside.
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # one decode step of one request that asks for its token's log probability and five others
        dict(name="logprobs_one", op="logprobs", t=1, vocab=32000, dtype="float32", k=5, asked=1.0),
        # a decode step of 64 requests, each with its own temperature and twenty alternatives
        dict(name="logprobs_step_64", op="logprobs", t=64, vocab=131072, dtype="bfloat16", k=20,
             asked=1.0, temperature=True),
        # windows of verified drafts, rejected ones not asked for, half the rows held to a grammar
        # that leaves a few tokens; an odd vocabulary
        dict(name="logprobs_guided_odd", op="logprobs", t=96, vocab=50001, dtype="float32", k=5,
             asked=0.7, guided=0.5),
        # scoring a prompt: every token's log probability, the best alternative beside it
        dict(name="logprobs_prompt_4k", op="logprobs", t=4096, vocab=131072, dtype="bfloat16", k=1,
             asked=1.0),
        # recording a teacher: 64 entries for each token, no token asked for; rows at odd addresses
        dict(name="logprobs_teacher_2k", op="logprobs", t=2048, vocab=50001, dtype="bfloat16", k=64,
             asked=-1.0),
        # the loss of one short sample
        dict(name="distill_small", op="distill", t=64, vocab=32000, dtype="bfloat16", k=8,
             tail=False, s=1.0, absent=0.0, padded=0.0),
        # an evaluation batch over a large vocabulary, the rest as one more outcome
        dict(name="distill_2k", op="distill", t=2048, vocab=131072, dtype="bfloat16", k=64,
             tail=True, s=1.0, absent=0.1, padded=0.1),
        # a gradient in fp32 over an odd vocabulary, tempered logits
        dict(name="distill_bwd_odd", op="distill_bwd", t=512, vocab=50001, dtype="float32", k=20,
             tail=False, s=0.5, absent=0.0, padded=0.1),
        # the gradient of the evaluation batch's size
        dict(name="distill_bwd_2k", op="distill_bwd", t=2048, vocab=131072, dtype="bfloat16", k=64,
             tail=True, s=1.0, absent=0.1, padded=0.1),
        # a step on a few tokens
        dict(name="distill_grad_small", op="distill_grad", t=16, vocab=32000, dtype="float32", k=16,
             tail=True, s=1.0, absent=0.0, padded=0.0),
        # a step on ragged samples: padded tokens, entries absent, logits a slice of wider rows
        dict(name="distill_grad_odd", op="distill_grad", t=1000, vocab=50001, dtype="bfloat16",
             k=32, tail=False, s=0.5, absent=0.2, padded=0.3, pad=175),
        # a training step on 4,096 tokens of a large vocabulary
        dict(name="distill_grad_4k", op="distill_grad", t=4096, vocab=131072, dtype="bfloat16",
             k=64, tail=True, s=1.0, absent=0.1, padded=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs", "distill", "distill_bwd", "distill_grad"])
    vocab, dtype = _log(rng, 500, 200000), rng.choice(["bfloat16", "bfloat16", "float32"])
    most = 4096 * 131072 * 2 // (vocab * (4 if dtype == "float32" else 2))
    c = dict(op=op, t=_log(rng, 1, min(4096, most)), vocab=vocab, dtype=dtype,
             pad=rng.choice([0, 0, 0, 1, 64, 333]))
    if op == "logprobs":
        return c | dict(k=rng.choice([0, 1, 5, rng.randint(1, 20), rng.randint(1, 128)]),
                        asked=rng.choice([1.0, 1.0, 0.6, -1.0]), guided=rng.choice([0.0, 0.0, 0.3]),
                        temperature=rng.random() < 0.5)
    return c | dict(k=_log(rng, 1, 256), tail=rng.random() < 0.5, s=rng.choice([1.0, 0.5, 0.8]),
                    absent=rng.choice([0.0, 0.1, 0.4]), padded=rng.choice([0.0, 0.2]))


def _kept(case, share, salt):
    """Which rows a call reads: the same for every seed, so that ``work`` can count them."""
    gen = torch.Generator().manual_seed(case["t"] * 31 + salt)
    kept = torch.rand(case["t"], generator=gen) < share
    kept[0] = True
    return kept


def work(case):
    t, v, k = case["t"], case["vocab"], case["k"]
    e = 4 if case["dtype"] == "float32" else 2
    if case["op"] == "logprobs":
        asked = case["asked"]
        rows = t if asked < 0 else int(_kept(case, asked, 1).sum())
        small = t * (4 + 8 * k) + (0 if asked < 0 else 8 * t) + (4 * t if case.get("temperature") else 0)
        return {"bytes": rows * v * e + small, "flops": 6 * rows * v}
    rows = int(_kept(case, 1 - case["padded"], 2).sum())
    small = t * 8 * k + (20 * t if case["op"] != "distill_grad" else 8 * t)
    back = 0 if case["op"] == "distill" else t * v * e
    return {"bytes": rows * v * e + back + small, "flops": 4 * rows * v}


# ------------------------------------------------------------------------------------ the inputs
def _logits(gen, case):
    """Rows of logits: a few dozen likely tokens over a broad floor, in rows `pad` wider than the
    vocabulary."""
    t, v = case["t"], case["vocab"]
    x = torch.randn(t, v + case.get("pad", 0), generator=gen, device=DEV) * 2
    few = min(48, v)
    at = torch.randint(0, v, (t, few), generator=gen, device=DEV)
    lift = 14 - 2.2 * torch.arange(1, few + 1, device=DEV).log()
    lift = lift + torch.randn(t, few, generator=gen, device=DEV)
    x.scatter_add_(1, at, lift * (0.4 + 0.6 * torch.rand(t, 1, generator=gen, device=DEV)))
    return x.to(getattr(torch, case["dtype"]))[:, :v]


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    t, v, k = case["t"], case["vocab"], case["k"]
    x = _logits(gen, case)
    s = dict(op=case["op"], x=x, k=k)
    if case["op"] == "logprobs":
        if case.get("guided"):
            held = torch.rand(t, 1, generator=gen, device=DEV) < case["guided"]
            few = torch.zeros(t, v, dtype=torch.bool, device=DEV)
            few.scatter_(1, torch.randint(0, v, (t, 4), generator=gen, device=DEV), True)
            x.masked_fill_(held & ~few, -math.inf)
        tokens = None
        if case["asked"] >= 0:  # drawn from the rows themselves
            race = x.float() - torch.empty(t, v, device=DEV).exponential_(generator=gen).log_()
            tokens = race.argmax(1).to(torch.int32)
            tokens[~_kept(case, case["asked"], 1).to(DEV)] = -1
        scale = None
        if case.get("temperature"):
            scale = 0.5 + torch.rand(t, generator=gen, device=DEV)
        return s | dict(tokens=tokens, scale=scale)
    # the teacher: another model's logits near the student's, its k largest log probabilities
    k = min(k, v - 1)
    z = x.float() + 0.7 * torch.randn(t, v, generator=gen, device=DEV)
    top, ids = torch.topk(z, k, dim=1)
    values = top - torch.logsumexp(z, 1, keepdim=True) if case["tail"] else top
    ids = ids.to(torch.int32)
    gone = torch.rand(t, k, generator=gen, device=DEV) < case["absent"]
    kept = _kept(case, 1 - case["padded"], 2).to(DEV)
    ids[gone | ~kept[:, None]] = -1
    values = torch.where(ids >= 0, values, -math.inf)
    # the mean over the tokens that count
    weight = torch.where(kept, 1.0 / kept.sum(), 0.0)
    if case["op"] == "distill_bwd":
        weight = weight * (0.5 + torch.rand(t, generator=gen, device=DEV))
    s |= dict(ids=ids, values=values, s=case["s"], tail=case["tail"], weight=weight)
    if case["op"] == "distill_bwd":  # what the forward call left
        s["stats"] = _loss(s)[1]
    return s


# ------------------------------------------------------------------------------- one pass of each
def run(s):
    if own:
        import kimi_delta_attention_03_gb300 as kda
        if s["op"] == "logprobs":
            return kda.token_logprobs(s["x"], s["tokens"], top_k=s["k"], inv_temperature=s["scale"])
        more = dict(inv_temperature=s["s"], tail=s["tail"])
        if s["op"] == "distill":
            return kda.distill_topk(s["x"], s["ids"], s["values"], **more)
        if s["op"] == "distill_bwd":
            return kda.distill_topk_bwd(s["weight"], s["x"], s["ids"], s["values"], s["stats"],
                                        **more)
        return kda.distill_topk_grad(s["x"], s["ids"], s["values"], s["weight"], **more)
    if s["op"] == "logprobs":
        return _logprobs(s)
    if s["op"] == "distill":
        return _loss(s)
    if s["op"] == "distill_bwd":
        return _grad(s, s["stats"])
    loss, stats = _loss(s)
    return loss, _grad(s, stats)


def _logprobs(s):
    x, tokens, k = s["x"].float(), s["tokens"], s["k"]
    t, v = x.shape
    scale = 1.0 if s["scale"] is None else s["scale"][:, None]
    m = x.amax(1, keepdim=True)
    y = (x - m) * scale
    e = torch.exp(y)
    total = e.sum(1)
    norm = total.log()
    entropy = norm - torch.where(e > 0, e * y, 0.0).sum(1) / total
    # the largest entries, the lowest index first among equals: one whole number for both
    bits = (x + 0.0).view(torch.int32)
    key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).to(torch.int64) << 32
    key = key + (v - 1 - torch.arange(v, device=x.device))
    n = min(k, v)
    ids = v - 1 - (torch.topk(key, n, dim=1).values & 0xFFFFFFFF)
    best = y.gather(1, ids) - norm[:, None]
    ids = torch.nn.functional.pad(ids, (0, k - n), value=-1)
    best = torch.nn.functional.pad(best, (0, k - n), value=-math.inf)
    ids = torch.where(best > -math.inf, ids, -1).to(torch.int32)
    if tokens is None:
        return None, entropy, ids, best
    live = tokens >= 0
    logprob = y.gather(1, tokens.clamp(min=0).long()[:, None])[:, 0] - norm
    return (torch.where(live, logprob, 0.0), torch.where(live, entropy, 0.0),
            torch.where(live[:, None], ids, -1), torch.where(live[:, None], best, -math.inf))


def _teacher(s):
    """Probabilities and log probabilities of the entries, what they leave, and their sum."""
    v = torch.where(s["ids"] >= 0, s["values"], -math.inf)
    if s["tail"]:
        rest = (1 - v.double().exp().sum(1)).clamp(min=0).float()
        p = v.exp()
        live = (s["ids"] >= 0).any(1)
        return p, v, rest, p.sum(1) + rest, live
    top = v.amax(1, keepdim=True)
    live = top[:, 0] > -math.inf
    v = v - torch.where(live[:, None], top, 0.0)
    e = v.exp()
    total = torch.where(live, e.sum(1), 1.0)[:, None]
    return e / total, v - total.log(), torch.zeros_like(total[:, 0]), live.float(), live


def _outside(s):
    """The logits without the teacher's tokens."""
    x = s["x"].float()
    t, v = x.shape
    at = torch.where(s["ids"] >= 0, s["ids"], v).long()
    held = torch.zeros(t, v + 1, dtype=torch.bool, device=x.device).scatter_(1, at, True)
    return torch.where(held[:, :v], -math.inf, x)


def _loss(s):
    x, scale = s["x"].float(), s["s"]
    p, logp, r, _, live = _teacher(s)
    m = x.amax(1)
    z = torch.exp((x - m[:, None]) * scale).sum(1)
    rest = _outside(s)
    mr = rest.amax(1)
    zr = torch.exp((rest - torch.where(mr > -math.inf, mr, 0.0)[:, None]) * scale).sum(1)
    y = (x.gather(1, s["ids"].clamp(min=0).long()) - m[:, None]) * scale - z.log()[:, None]
    loss = torch.where(p > 0, p * (logp - y), 0.0).sum(1)
    yr = (mr - m) * scale + zr.log() - z.log()
    loss = loss + torch.where(r > 0, r * (r.log() - yr), 0.0)
    stats = torch.stack([m, z, mr, zr], 1)
    return torch.where(live, loss, 0.0), torch.where(live[:, None], stats, 0.0)


def _grad(s, stats):
    x, scale = s["x"].float(), s["s"]
    t, v = x.shape
    p, _, r, total, live = _teacher(s)
    m, z, mr, zr = stats[:, :, None].unbind(1)
    d = torch.exp((x - m) * scale) * (total[:, None] / z)
    if s["tail"]:
        mr = torch.where(mr > -math.inf, mr, 0.0)
        share = torch.where(zr > 0, r[:, None] / zr, 0.0)
        d = d - torch.exp((_outside(s) - mr) * scale) * share
    at = torch.where(s["ids"] >= 0, s["ids"], v).long()
    d = torch.nn.functional.pad(d, (0, 1)).scatter_add_(1, at, -p)[:, :v]
    d = d * (s["weight"] * scale)[:, None]
    on = live & (s["weight"] != 0)
    return torch.where(on[:, None], d, 0.0).to(s["x"].dtype)


# ---------------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    rows = max(1, (1 << 25) // case["vocab"])
    each = _exact_logprobs if case["op"] == "logprobs" else _exact_distill
    parts = [each(s, slice(i, i + rows)) for i in range(0, case["t"], rows)]
    got = [None if c[0] is None else torch.cat(c) for c in zip(*parts)]
    if case["op"] == "logprobs":
        return tuple(got)
    loss, stats, grad = got
    return {"distill": (loss, stats), "distill_bwd": grad, "distill_grad": (loss, grad)}[case["op"]]


def _exact_logprobs(s, at):
    """log softmax of the tempered rows, its entropy, its largest entries."""
    x = s["x"][at].double()
    y = x if s["scale"] is None else x * s["scale"][at].double()[:, None]
    logq = torch.log_softmax(y, 1)
    entropy = torch.special.entr(logq.exp()).sum(1)
    k = s["k"]
    order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k]
    best = logq.gather(1, order)
    order = torch.where(best == -math.inf, -1, order).to(torch.int32)
    short = k - order.shape[1]
    if short:
        order = torch.cat([order, order.new_full((len(x), short), -1)], 1)
        best = torch.cat([best, best.new_full((len(x), short), -math.inf)], 1)
    if s["tokens"] is None:
        return None, entropy, order, best
    tokens = s["tokens"][at].long()
    off = tokens < 0
    logprob = logq.gather(1, tokens.clamp(min=0)[:, None])[:, 0]
    return (logprob.masked_fill(off, 0), entropy.masked_fill(off, 0),
            order.masked_fill(off[:, None], -1), best.masked_fill(off[:, None], -math.inf))


def _exact_distill(s, at):
    """KL between the two distributions over the entries (and the rest), and its derivative."""
    x, scale = s["x"][at].double(), s["s"]
    ids, v = s["ids"][at].long(), s["values"][at].double()
    there = ids >= 0
    v = v.masked_fill(~there, -math.inf)
    logq = torch.log_softmax(x * scale, 1)
    q = logq.exp()
    held = torch.zeros_like(x)
    held.scatter_add_(1, ids.clamp(min=0), there.double())
    held = held > 0
    if s["tail"]:
        live = there.any(1)
        logp, p = v, v.exp()
        r = (1 - p.sum(1)).clamp(min=0)
    else:
        live = (v > -math.inf).any(1)
        logp = torch.log_softmax(v.masked_fill(~live[:, None], 0), 1)
        p = logp.exp()
        r = torch.zeros_like(p[:, 0])
    mass = p.sum(1) + r
    logr = torch.logsumexp((x * scale).masked_fill(held, -math.inf), 1) - torch.logsumexp(x * scale, 1)
    loss = torch.where(p > 0, p * (logp - logq.gather(1, ids.clamp(min=0))), 0).sum(1)
    loss = loss + torch.where(r > 0, r * (r.log() - logr), 0)
    d = mass[:, None] * q
    d.scatter_add_(1, ids.clamp(min=0), torch.where(there, -p, 0))
    d = d - torch.where(held, 0, (r / logr.exp()).nan_to_num(0, 0, 0)[:, None] * q)
    g = s["weight"][at].double() * scale
    d = d * g[:, None]
    rest = x.masked_fill(held, -math.inf)
    m, mr = x.amax(1), rest.amax(1)
    z = ((x - m[:, None]) * scale).exp().sum(1)
    zr = ((rest - mr[:, None]) * scale).exp().sum(1)
    stats = torch.stack([m, z, mr, zr], 1)
    off = ~live
    return loss.masked_fill(off, 0), stats.masked_fill(off[:, None], 0), d.masked_fill(off[:, None], 0)
