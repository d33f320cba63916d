"""Plain implementations in 64 bits of the operators over vocabulary rows, and how far fp32 may be off.

The bounds.  u = 2^-24 is half a step of fp32, relative.  An exponential's argument (x - m) s log2(e) takes
two roundings and a constant rounded once, so a weight with |a| octaves is off by at most 3 u |a| ln 2, and
by 2^-22 more for the approximate exponential: its absolute error against the largest weight is below
2^-21, whatever a.  What these errors add to z relative to z is at most 2^-22 + 3 u E|ln weight|, and E|ln
weight| <= ln V + entropy-like terms <= 2 ln V.  A thread sums at most V / 1024 + 16 weights one after
another (512 threads with two sums each, 256 with two sums each over at least half as many CTAs), and
log2(4096) levels of joining follow.
"""
import math

import torch

U = 2.0 ** -24


def step(dtype):
    """Half a step of the type, relative."""
    return torch.finfo(dtype).eps / 2


def sum_error(vocab):
    """Relative error of z, and with it absolute of its logarithm."""
    return 2.0 ** -22 + 3 * U * 2 * math.log(vocab + 1) + U * (vocab / 512 + 64)


def logprobs(x, tokens, k, scale=None):
    """(logprob, entropy, ids, best) as token_logprobs gives them, for rows of finite and -inf logits."""
    x = x.double()
    y = x if scale is None else x * scale.double()[:, None]
    t, v = x.shape
    m = y.amax(1, keepdim=True)
    logq = y - m - (y - m).exp().sum(1, keepdim=True).log()
    q = logq.exp()
    entropy = -torch.where(q > 0, q * logq, 0.0).sum(1)
    ids = torch.full((t, k), -1, dtype=torch.int32)
    best = torch.full((t, k), -math.inf, dtype=torch.float64)
    order = torch.sort(x + 0.0, dim=1, descending=True, stable=True).indices[:, :k]
    there = x.gather(1, order) > -math.inf
    ids[:, :min(k, v)] = torch.where(there, order, -1).to(torch.int32)
    best[:, :min(k, v)] = torch.where(there, logq.gather(1, order), -math.inf)
    if tokens is None:
        return None, entropy, ids, best
    off = tokens < 0
    logprob = logq.gather(1, tokens.clamp(min=0).long()[:, None])[:, 0]
    return (logprob.masked_fill(off, 0), entropy.masked_fill(off, 0), ids.masked_fill(off[:, None], -1),
            best.masked_fill(off[:, None], -math.inf))


def distill(x, ids, values, scale, tail):
    """dict of loss [T], its gradient grad [T, V], their bounds loss_error and grad_error, and stats."""
    x, values = x.double(), values.double()
    t, v = x.shape
    loss, stats = torch.zeros(t, dtype=torch.float64), torch.zeros(t, 4, dtype=torch.float64)
    grad, grad_error = torch.zeros(t, v, dtype=torch.float64), torch.zeros(t, v, dtype=torch.float64)
    loss_error = torch.zeros(t, dtype=torch.float64)
    e = sum_error(v)
    for i in range(t):
        entries = [(int(a), float(b)) for a, b in zip(ids[i], values[i]) if 0 <= a < v]
        if not entries or (not tail and all(b == -math.inf for _, b in entries)):
            continue
        val = torch.tensor([b for _, b in entries], dtype=torch.float64)
        at = torch.tensor([a for a, _ in entries])
        logp = val if tail else val - torch.logsumexp(val, 0)
        p = logp.exp()
        r = max(0.0, 1 - float(p.sum())) if tail else 0.0
        y = x[i] * scale
        m = float(x[i].max())
        logq = y - m * scale - ((x[i] - m) * scale).exp().sum().log()
        q = logq.exp()
        out = torch.ones(v, dtype=torch.bool)
        out[at] = False
        rest = x[i][out]
        mr = float(rest.max()) if len(rest) else -math.inf
        zr = float(((rest - mr) * scale).exp().sum()) if mr > -math.inf else 0.0
        z = float(((x[i] - m) * scale).exp().sum())
        stats[i] = torch.tensor([m, z, mr, zr], dtype=torch.float64)
        terms = torch.where(p > 0, p * (logp - logq[at]), 0.0)
        # each difference is formed from three values, each rounded; p within 2^-20 of itself
        size = torch.where(p > 0, p * (logp.abs() + logq[at].abs() + abs(m * scale) + 1), 0.0).sum()
        loss[i] = terms.sum()
        loss_error[i] = e * p.sum() + 2.0 ** -20 * size
        mass = float(p.sum()) + r
        held = torch.zeros(v, dtype=torch.float64).scatter_add_(0, at, p)
        d = mass * q - held
        big = mass * q + held
        if r > 0:
            if zr > 0:
                logqr = (mr - m) * scale + math.log(zr / z)
                loss[i] += r * (math.log(r) - logqr)
                loss_error[i] += e * r * 2 + 2.0 ** -20 * r * (abs(math.log(r)) + abs(logqr) + abs(m * scale) + 1)
                share = torch.where(out, r * (logq - logqr).exp(), 0.0)
                d, big = d - share, big + share
            else:
                loss[i] = math.inf
        grad[i] = d * scale
        # a weight of 126 octaves is within 3 u 126 ln 2 < 2^-15.  Below 2^-126 it is flushed to zero, and its
        # factor scale (mass / z + r / zr) is at most 2 scale mass, as z and zr hold their largest weight, 1
        grad_error[i] = big * scale * (2 * e + 2.0 ** -15) + scale * mass * 2.0 ** -125
    return dict(loss=loss, grad=grad, loss_error=loss_error, grad_error=grad_error, stats=stats)
