"""The splits of queries and softmax weights restated with torch's conversions on the CPU: a bf16 as
e4m3 plus e5m2, and an f16 weight p = P0 + P1 / 2^5 + P2 / 2^10 in e4m3, the last term rounded from a
place that depends on the key.  What the attention call states of them follows from the formats."""
import numpy as np
import pytest
import torch

PEAK = 2.0 ** 6  # a weight at its row's reference; weights go up to 2^8


def e4m3(x):
    assert x.abs().max() <= 448
    return x.float().to(torch.float8_e4m3fn).to(torch.float16)


def places():
    """Of the 128 keys of a tile, in units of P2."""
    rev = torch.tensor([int(f"{k:07b}"[::-1], 2) for k in range(128)])
    return ((2 * rev - 127) * 15).double() * 2.0 ** -21


def held(x, place):
    p = x.to(torch.float16)
    p0 = e4m3(p)
    d1 = (p - p0) * 32
    p1 = e4m3(d1)
    p2 = e4m3(((d1 - p1).double() * 32 + place).to(torch.float16))
    return p0.double() + p1.double() / 32 + p2.double() / 1024


@pytest.mark.parametrize("octave", range(-2, 27))
def test_weights_keep_what_the_call_states(octave):
    """Weights of 2^-octave of the largest and up to an octave less: 11 bits (half a step is 2^-11 of
    the weight or less) down to 2^-15, 2^-25 of the largest below; 2^-29 on average over a tile."""
    x = PEAK * torch.exp2(-octave - torch.linspace(0, 1, 3001, dtype=torch.float64))
    err = torch.stack([held(x, float(t)) - x for t in places()])
    each = x * 2.0 ** -11 if octave < 15 else torch.full_like(x, PEAK * 2.0 ** -25)
    assert (err.abs() <= each).all()
    assert (err.mean(0).abs() <= x * 2.0 ** -11 + PEAK * 2.0 ** -29).all()


def test_weights_that_the_terms_can_hold_are_exact():
    """Every f16 from 2^-15 of the largest up, at every key's place, and zero."""
    p = torch.arange(0, 0x7C00, dtype=torch.int32).to(torch.int16).view(torch.float16)
    p = p[(p == 0) | ((p >= PEAK * 2.0 ** -15) & (p <= 256))]
    for t in places():
        assert torch.equal(held(p, float(t)), p.double())


def test_places_are_even_and_keep_exact_terms():
    t = places().numpy()
    assert np.allclose(np.diff(np.sort(t)), 15 * 2.0 ** -20) and abs(t.sum()) < 1e-12
    assert np.abs(t).max() < 2.0 ** -10 and (t.astype(np.float16) == t).all()


def test_the_two_terms_of_a_query_restated():
    """Every bf16 below 2^8 as e4m3 plus e5m2, as the rows of q are held (largest in [2^7, 2^8))."""
    q = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).float()
    q = q[q.abs() < 256]
    hi = q.to(torch.float8_e4m3fn).float()
    off = (hi + (q - hi).to(torch.float8_e5m2).float() - q).abs()
    assert (off[q.abs() >= 2.0 ** -5] == 0).all() and off.max() <= 2.0 ** -14
