"""Bounds for the operators over vocabulary rows from the values that the kernels form, and 64-bit definitions
that run on the inputs' device, for tests of many rows.

u = 2^-24 is half a step of fp32, relative; ex2.approx adds 2^-22.

z, the sum of a row's weights.  A weight of a octaves has an argument from two roundings and a constant rounded
once, so it is off by at most 3 u |a| ln 2 of itself; over the row that is at most 3 u E|ln weight| <= 6 u ln V.
A row has at least one CTA of `threads` threads (256, or 128 for many short rows); each adds its V / threads
entries to two sums, V / (2 threads) additions one after another, and up to two dozen roundings of the edges'
entries, raised references and levels of joining follow.

Losses: sum_i p_i (logp_i - ((x_i - m) s - ln z)) + r (ln r - ((m_r - m) s + ln z_r - ln z)).
  D = (x - m) s takes two roundings: 2 u |D|.  ln z is off by z's relative error, 2 u |ln z| of the logarithm
  itself.  The two differences around it: 2 u (|logp| + |D| + |ln z|).
  p: with tail expf of a given value, 4 u p.  Else expf(d) / z_t, d = v - max rounded to u |d|, |d| <= |logp|,
  and z_t a sum of at most 256 weights; logp = d - ln z_t is off by u |d| + e_t + 3 u |logp|.
  The sum: five levels of a warp's, eight warps one after another, 14 u of the terms' sizes.
  Together below 32 u p (|logp| + |D| + |ln z| + 1), the product of p's error u |logp| with the term, and e_t.
  r is 1 less a sum of integers in units of 2^-40, each exponential within 2^-30: within 2^-29 and its rounding.
"""
import math

import torch

U = 2.0 ** -24


def sum_error(vocab, threads=256):
    """Relative error of z, and with it absolute of its logarithm."""
    return 2.0 ** -22 + 6 * U * math.log(vocab + 1) + U * (vocab / (2 * threads) + 64)


def distill(x, ids, values, scale, tail):
    """dict of loss [T], its gradient grad [T, V] and their bounds loss_error and grad_error, in 64 bits; scale is
    a value of fp32.  Every row has a distribution and some tokens that no entry names, with a finite logit."""
    x, v = x.double(), values.double()
    t, vocab = x.shape
    e, e_t = sum_error(vocab), 0.0 if tail else sum_error(256)
    there = ids >= 0
    at = torch.where(there, ids, vocab).long()
    v = torch.where(there, v, -math.inf)
    live = there.any(1) if tail else (v > -math.inf).any(1)
    logp = v if tail else torch.log_softmax(v.masked_fill(~live[:, None], 0), 1)
    p = torch.where(there, logp.exp(), 0.0)
    r = (1 - p.sum(1)).clamp(min=0) if tail else torch.zeros_like(p[:, 0])
    mass = p.sum(1) + r
    named = torch.zeros(t, vocab + 1, dtype=torch.bool, device=x.device).scatter_(1, at, True)[:, :vocab]
    rest = x.masked_fill(named, -math.inf)
    m, mr = x.amax(1), rest.amax(1)
    w = ((x - m[:, None]) * scale).exp()
    wr = ((rest - mr[:, None]) * scale).exp()
    lz, lzr = w.sum(1).log(), wr.sum(1).log()
    q = w / w.sum(1, keepdim=True)
    # the entries
    d = (torch.nn.functional.pad(x, (0, 1)).gather(1, at) - m[:, None]) * scale
    gap = logp - (d - lz[:, None])
    counts = p > 0
    loss = torch.where(counts, p * gap, 0.0).sum(1)
    size = logp.abs() + d.abs() + lz[:, None].abs() + 1
    own = 32 * U * size + (U * logp.abs() + e_t) * gap.abs() + e + e_t
    error = torch.where(counts, p * own, 0.0).sum(1)
    # the tokens outside
    dr = (mr - m) * scale
    dr_size = r.log().clamp(min=-21).abs() + dr.abs() + lzr.abs() + lz.abs() + 1
    loss = loss + torch.where(r > 0, r * (r.log() - (dr + lzr - lz)), 0.0)
    if tail:
        error = error + 2 * (2.0 ** -29 + U * r) * (dr_size + 1) + r * (2 * e + 32 * U * dr_size)
    # the gradient: a weight of a octaves, |a| at most 126, within 3 u |a| ln 2; below they are zeros
    # p as above, entries of one token added one after another
    zeros = torch.zeros(t, vocab + 1, dtype=torch.float64, device=x.device)
    given = zeros.scatter_add(1, at, p)[:, :vocab]
    p_error = torch.where(counts, p * ((32 + ids.shape[1]) * U + U * logp.abs() + e_t), 0.0)
    given_error = zeros.scatter_add(1, at, p_error)[:, :vocab]
    share = torch.where(named, 0.0, (r / wr.sum(1))[:, None] * wr)
    grad = scale * (mass[:, None] * q - given - share)
    slack = (2 * e + 2.0 ** -15) * (mass[:, None] * q + share) + given_error
    slack = scale * slack + scale * mass[:, None] * 2.0 ** -125
    if tail:  # what r is off by, in its share
        slack = slack + scale * torch.where(named, 0.0, 2.0 ** -29 / wr.sum(1)[:, None] * wr)
    off = ~live
    return dict(loss=loss.masked_fill(off, 0), loss_error=error.masked_fill(off, 0),
                grad=grad.masked_fill(off[:, None], 0), grad_error=slack.masked_fill(off[:, None], 0))
