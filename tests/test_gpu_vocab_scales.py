"""Logits whose differences are beyond fp32, at inverse temperatures that bring them back into its range."""
import math

import pytest
import torch

from tests import vocab_bounds as bounds
from tests import vocab_reference as ref
from tests.test_gpu_vocab import BF16, DEV, F32, INF, gen, kda
from tests.test_gpu_vocab_bounds import check


def vast(seed, t, v, dtype):
    """Entries of either sign up to the type's largest."""
    x = (torch.rand(t, v, generator=gen(seed)).double() * 2 - 1) * 3.3e38
    x[:, 1], x[:, v // 2] = torch.finfo(dtype).max, torch.finfo(dtype).min
    return x.to(dtype)


SCALES = [2e-38, 3e-37, 1e-30, 1e-12, 0.25]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("t,v", [(5, 9001), (5, 17), (700, 5003)])
def test_logprobs_of_vast_logits(dtype, t, v):
    x = vast(1, 5, v, dtype)
    scale = torch.tensor(SCALES)
    tokens = torch.full((5,), v // 2, dtype=torch.int32)
    want = ref.logprobs(x, tokens, 7, scale)
    n = t // 5
    got = kda().token_logprobs(x.to(DEV).repeat(n, 1), tokens.to(DEV).repeat(n), top_k=7,
                               inv_temperature=scale.to(DEV).repeat(n))
    e = bounds.sum_error(v, 128)
    for i in range(n):
        lp, entropy, ids, best = (a[5 * i:5 * i + 5].cpu() for a in got)
        assert torch.equal(ids, want[2])
        for a, b in ((lp, want[0]), (best, want[3])):
            assert a.isfinite().all() and b.isfinite().all()
            # (x - m) s: two roundings; ln z: e and its own two; their difference: one
            assert float(((a.double() - b).abs() - 4 * bounds.U * b.abs()).max()) <= e + 4 * bounds.U * math.log(v + 1)
        assert float((entropy.double() - want[1]).abs().max()) <= (3 * e + 2.0 ** -20) * (1 + math.log(v + 1))
    assert kda().read_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("scale", SCALES)
def test_distillation_of_vast_logits(dtype, tail, scale):
    """The weights are large, so that gradients of tiny scales are no subnormal values."""
    scale = float(torch.tensor(scale))
    x = vast(2, 4, 9001, dtype)
    ids = torch.randint(0, 9001, (4, 12), generator=gen(3), dtype=torch.int32)
    ids[:, 0], ids[:2, 1] = 1, 9001 // 2
    ids[:, 2:] = torch.stack([torch.randperm(3000, generator=gen(i))[:10] + 10 for i in range(4)]).to(torch.int32)
    val = torch.log_softmax(torch.randn(4, 20, generator=gen(4)), 1)[:, :12]
    weight = (torch.rand(4, generator=gen(5)) + 0.5) * (2.0 ** 100 if scale < 1e-20 else 1.0)
    assert INF > float(weight.max())
    check(x.to(DEV), ids.to(DEV), val.to(DEV), scale, tail, weight.to(DEV))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_logprobs_at_the_ends_of_the_inverse_temperatures(dtype):
    """From fp32's smallest subnormal value to 2^127; above it, as where it is not positive, a row gets NaN."""
    v = 3001
    scale = torch.tensor([1e-45, 1e-40, 1e-38, 2.0 ** 126, 2.0 ** 127, math.nextafter(2.0 ** 127, 1e40) * 1.001, 3.4e38,
                          INF, -1e-45])
    x = vast(6, 9, v, dtype)
    tokens = torch.full((9,), 1, dtype=torch.int32)
    got = [a.cpu() for a in kda().token_logprobs(x.to(DEV), tokens.to(DEV), top_k=5, inv_temperature=scale.to(DEV))]
    lp, entropy, ids, best = got
    for a in (lp, entropy, best):
        assert a[5:].isnan().all() and not a[:5].isnan().any()
    assert (ids[5:] == -1).all()
    want = ref.logprobs(x[:5], tokens[:5], 5, scale[:5])
    assert torch.equal(ids[:5], want[2])
    # as above, and a subnormal s log2(e) is off by 2^-150, times differences below 2^129
    e = bounds.sum_error(v) + 2.0 ** -21
    for a, b in ((lp[:5], want[0]), (best[:5], want[3])):
        beyond = b.float() == -INF
        assert torch.equal(a == -INF, beyond)
        off = torch.where(beyond, 0.0, (a.double() - b).abs() - 4 * bounds.U * b.abs())
        assert float(off.max()) <= e + 4 * bounds.U * math.log(v + 1)
    assert float((entropy[:5].double() - want[1]).abs().max()) <= (3 * e + 2.0 ** -20) * (1 + math.log(v + 1))
    assert kda().read_device_status() == 0
