"""Host-side refusals of the vocabulary calls, and pins of the plain implementations that the GPU tests
compare with.  No GPU needed: every call below is rejected or answered on the host."""
import math

import pytest
import torch

from tests import vocab_reference as ref

OK, INVALID, UNSUPPORTED = 0, -1, -2
P = 1 << 20  # a made-up device address: nothing is launched with it


@pytest.fixture(scope="module")
def lib():
    from kimi_delta_attention_03_gb300 import build, binding
    build.build()
    return binding.load_library()


@pytest.mark.parametrize("want,kw", [
    (OK, dict(t=0)), (INVALID, dict(t=-1)), (INVALID, dict(v=0)), (INVALID, dict(k=-1)),
    (UNSUPPORTED, dict(t=2 ** 31)), (UNSUPPORTED, dict(v=2 ** 30 + 1, stride=2 ** 31)),
    (UNSUPPORTED, dict(k=129)), (UNSUPPORTED, dict(dtype=2)), (UNSUPPORTED, dict(dtype=99)),
    (INVALID, dict(x=None)), (INVALID, dict(x=P + 2)), (INVALID, dict(x=P + 1, dtype=0)),
    (INVALID, dict(stride=9)), (INVALID, dict(lp=None)), (INVALID, dict(entropy=None)),
    (INVALID, dict(ids=None)), (INVALID, dict(best=None))])
def test_logprobs_refuses(lib, want, kw):
    a = dict(t=3, v=10, dtype=1, x=P, stride=10, tokens=P, scale=None, k=2, lp=P, entropy=P, ids=P, best=P) | kw
    assert lib.kda_token_logprobs(*a.values(), None) == want


BASE = dict(t=3, v=10, dtype=1, x=P, stride=10, k=2, ids=P, val=P, s=1.0, tail=0)
COMMON = [
    (OK, dict(t=0)), (INVALID, dict(t=-1)), (INVALID, dict(v=0)), (INVALID, dict(k=0)),
    (INVALID, dict(tail=2)), (INVALID, dict(tail=-1)), (INVALID, dict(tail=1, k=10)), (INVALID, dict(s=0.0)),
    (INVALID, dict(s=-1.0)), (INVALID, dict(s=math.inf)), (INVALID, dict(s=math.nan)), (INVALID, dict(s=2e30)),
    (UNSUPPORTED, dict(k=257)), (UNSUPPORTED, dict(t=2 ** 28)), (UNSUPPORTED, dict(dtype=2)),
    (UNSUPPORTED, dict(v=393217, stride=393217)), (UNSUPPORTED, dict(v=786433, stride=786433, dtype=0)),
    (INVALID, dict(x=None)), (INVALID, dict(x=P + 2)), (INVALID, dict(ids=None)), (INVALID, dict(val=None)),
    (INVALID, dict(stride=9))]


@pytest.mark.parametrize("want,kw", COMMON + [
    (INVALID, dict(loss=None)), (INVALID, dict(stats=None)), (INVALID, dict(stats=P + 8))])
def test_distill_refuses(lib, want, kw):
    a = BASE | dict(loss=P, stats=P) | kw
    assert lib.kda_distill_topk(*a.values(), None) == want


@pytest.mark.parametrize("want,kw", COMMON + [
    (INVALID, dict(stats=None)), (INVALID, dict(stats=P + 8)), (INVALID, dict(w=None)), (INVALID, dict(d=None)),
    (INVALID, dict(d=P + 2)), (INVALID, dict(ds=9)), (INVALID, dict(d=P, ds=12))])
def test_distill_bwd_refuses(lib, want, kw):
    a = BASE | dict(stats=P, w=P, d=P + 4096, ds=10) | kw
    assert lib.kda_distill_topk_bwd(*a.values(), None) == want


@pytest.mark.parametrize("want,kw", COMMON + [
    (INVALID, dict(loss=None)), (INVALID, dict(w=None)), (INVALID, dict(d=None)), (INVALID, dict(d=P + 2)),
    (INVALID, dict(ds=9)), (INVALID, dict(d=P, ds=12))])
def test_distill_grad_refuses(lib, want, kw):
    a = BASE | dict(w=P, loss=P, d=P + 4096, ds=10) | kw
    assert lib.kda_distill_topk_grad(*a.values(), None) == want


def test_reference_log_probabilities():
    ln = math.log
    x = torch.tensor([[ln(1), ln(2), ln(5)], [0.0, -math.inf, 0.0]], dtype=torch.float64)
    lp, entropy, ids, best = ref.logprobs(x, torch.tensor([1, 2], dtype=torch.int32), 3)
    assert torch.allclose(lp, torch.tensor([ln(0.25), ln(0.5)], dtype=torch.float64))
    h = -(ln(1 / 8) / 8 + ln(1 / 4) / 4 + 5 * ln(5 / 8) / 8)
    assert torch.allclose(entropy, torch.tensor([h, ln(2)], dtype=torch.float64))
    assert ids.tolist() == [[2, 1, 0], [0, 2, -1]]
    assert best[1].tolist() == [ln(0.5), ln(0.5), -math.inf]
    x = torch.randint(-2, 3, (7, 300), generator=torch.Generator().manual_seed(2)).float()
    x = torch.where((x == 0) & (torch.arange(300) % 3 == 0), -0.0, x)
    for row, got in zip(x, ref.logprobs(x, None, 40)[2]):
        assert got.tolist() == sorted(range(300), key=lambda j: (-float(row[j]), j))[:40]


@pytest.mark.parametrize("tail", [False, True])
def test_reference_distillation_is_the_divergence_and_its_derivative(tail):
    g = torch.Generator().manual_seed(1)
    x = torch.randn(4, 9, generator=g, dtype=torch.float64)
    z = torch.randn(4, 9, generator=g, dtype=torch.float64)
    val, ids = torch.topk(torch.log_softmax(z, 1), 3, dim=1)
    x.requires_grad_(True)
    logq = torch.log_softmax(0.7 * x, 1)
    if tail:
        keep = torch.zeros(4, 9, dtype=torch.bool).scatter_(1, ids, True)
        p = torch.softmax(z, 1)
        r, qr = (p * ~keep).sum(1), (logq.exp() * ~keep).sum(1)
        loss = (val.exp() * (val - logq.gather(1, ids))).sum(1) + r * (r.log() - qr.log())
    else:
        p = torch.softmax(val, 1)
        loss = torch.nn.functional.kl_div(logq.gather(1, ids), p, reduction="none").sum(1)
    loss.sum().backward()
    got = ref.distill(x.detach(), ids, val, 0.7, tail)
    assert torch.allclose(got["loss"], loss.detach()) and torch.allclose(got["grad"], x.grad)
    # a student that is the teacher has no loss and no gradient
    if tail:
        got = ref.distill(z, ids, val, 1.0, True)
        assert float(got["loss"].abs().max()) < 1e-14 and float(got["grad"].abs().max()) < 1e-14
