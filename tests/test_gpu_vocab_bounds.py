"""The vocabulary calls within bounds from the values that their kernels form: losses of rows far from zero,
every entry of many large rows, and the many short rows that CTAs of 128 threads take."""
import math

import pytest
import torch

from tests import vocab_bounds as bounds
from tests import vocab_reference as ref
from tests.test_gpu_vocab import BF16, DEV, F32, INF, gen, kda, logits, teacher


def close(got, want, error):
    assert torch.equal(got.isinf(), want.isinf()) and not got.isnan().any()
    off = torch.where(want.isinf(), 0.0, (got.double() - want).abs() - error)
    assert float(off.max()) <= 0, (float(off.max()), int(off.argmax()))


def check(x, ids, val, scale, tail, weight):
    """All three calls on rows on the GPU."""
    want = bounds.distill(x, ids, val, scale, tail)
    loss, stats = kda().distill_topk(x, ids, val, scale, tail)
    close(loss, want["loss"], want["loss_error"])
    w = weight.double()[:, None]
    half = ref.step(x.dtype)
    grad = want["grad"] * w
    error = want["grad_error"] * w.abs() * (1 + half) + half * grad.abs() + 2.0 ** -133
    close(kda().distill_topk_bwd(weight, x, ids, val, stats, scale, tail), grad, error)
    loss, d = kda().distill_topk_grad(x, ids, val, weight, scale, tail)
    close(loss, want["loss"], want["loss_error"])
    close(d, grad, error)
    assert kda().read_device_status() == 0
    return loss


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("scale", [2.0 ** -20, 0.5, 1.0, 30.0, 1e6])
def test_losses_of_rows_far_from_zero(dtype, tail, scale):
    """A row moved as a whole has the same loss: within the bound that knows nothing of how far it is."""
    scale = float(torch.tensor(scale))
    x = logits(50, 6, 9001, F32, spread=1.0)
    x = ((x * 16).round() / 16).clamp(-15, 15)     # of which a bf16 or fp32 value holds what is moved, too
    ids, val = teacher(51, x, 10, True)
    weight = 0.5 + torch.rand(6, generator=gen(52))
    by = torch.tensor([0.0, 3e4, -3e4, 2.0 ** 18, -2.0 ** 19, 4096.0])[:, None]
    if dtype is BF16:  # 8 bits: multiples of 1 up to 128, 16 among 2^11 ..
        x, by = x.round(), torch.tensor([0.0, 112.0, -112.0, 64.0, -64.0, 100.0])[:, None]
    y = (x + by).to(dtype)
    assert torch.equal(y.double() - by.double(), x.double())
    args = [a.to(DEV) for a in (ids, val)]
    want = bounds.distill(x.to(DEV), *args, scale, tail)
    got = check(y.to(DEV), *args, scale, tail, weight.to(DEV))
    close(got, want["loss"], want["loss_error"])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,t,v", [(BF16, 620, 90007), (F32, 620, 45001), (BF16, 1300, 70001)])
def test_every_entry_of_many_large_rows(dtype, t, v):
    """More rows than are under way at a time, parts that are read again backwards: every row and entry of all
    three calls, with weights at which the smallest entries count."""
    g = torch.Generator(device=DEV).manual_seed(v)
    few = 20
    x = (torch.randn(t, v, generator=g, device=DEV) * 2).to(dtype)
    ids, val = teacher(60, x[:few].cpu(), 40, True, absent=0.1)
    ids, val = (a[torch.arange(t) % few].to(DEV) for a in (ids, val))
    weight = torch.rand(t, generator=gen(61)).to(DEV) + 0.5
    loss, stats = kda().distill_topk(x, ids, val, 1.0, True)
    alone = kda().distill_topk_bwd(weight, x, ids, val, stats, 1.0, True)
    loss2, both = kda().distill_topk_grad(x, ids, val, weight, 1.0, True)
    half = ref.step(dtype)
    for i in range(0, t, 155):
        rows = slice(i, i + 155)
        want = bounds.distill(x[rows], ids[rows], val[rows], 1.0, True)
        w = weight[rows].double()[:, None]
        grad = want["grad"] * w
        error = want["grad_error"] * w * (1 + half) + half * grad.abs() + 2.0 ** -133
        for got in (alone, both):
            close(got[rows], grad, error)
        # the bound tells an entry from zero, but for those whose two terms cancel
        assert float((error < grad.abs() / 2).float().mean()) > 0.9
        for got in (loss, loss2):
            close(got[rows], want["loss"], want["loss_error"])
    assert kda().read_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,v", [(BF16, 32760), (BF16, 32768), (BF16, 20011), (F32, 16381), (F32, 16384)])
@pytest.mark.parametrize("k", [1, 20, 64])
def test_many_short_rows(dtype, v, k):
    """Up to 64 KB a row, above 608 of them: CTAs of 128 threads, four batches a thread and more, with rows of
    equal entries by the thousand among them."""
    g = gen(v + k)
    x = logits(v + k, 20, v, dtype)
    low = torch.finfo(dtype).min
    few = torch.zeros(20, v, dtype=torch.bool).scatter_(1, torch.randint(0, v, (20, 4), generator=g), True)
    for row, mask in ((0, low), (1, -1e9), (2, -1e4), (3, -65504.0), (4, -INF)):
        x[row] = torch.where(few[row], x[row], torch.tensor(mask, dtype=dtype))
    x[5] = low
    x[6] = -1.5
    x[6, v - 3:] = 2.0
    x[7] = torch.where(torch.arange(v) < v // 2, -7.0, 0.1).to(dtype)
    x[8, v // 2:] = torch.randint(0, 2, (v - v // 2,), generator=g).to(dtype)
    x[9] = torch.linspace(-9, 9, v).to(dtype)
    x[10] = x[9].flip(0)
    tokens = torch.randint(-1, v, (20,), generator=g, dtype=torch.int32)
    tokens[5] = v - 1
    scale = 0.25 + torch.randint(1, 8, (20,), generator=g) / 4
    want = ref.logprobs(x, tokens, k, scale)
    got = kda().token_logprobs(x.to(DEV).repeat(31, 1), tokens.to(DEV).repeat(31), top_k=k,
                               inv_temperature=scale.to(DEV).repeat(31))
    e = bounds.sum_error(v, 128)
    u = bounds.U
    for i in range(31):
        lp, entropy, ids, best = (a[20 * i:20 * i + 20].cpu() for a in got)
        assert torch.equal(ids, want[2])
        for a, b in ((lp, want[0]), (best, want[3])):
            # (x - m) s: two roundings; ln z: e and its own two; their difference: one.  What is beyond fp32 (a
            # mask's lowest value, -(2 - 2^-7) 2^127, times a scale of 1.25 or more) is -inf as an fp32 value.
            beyond = b.float() == -INF
            assert torch.equal(a == -INF, beyond)
            off = torch.where(beyond, 0.0, (a.double() - b).abs() - 4 * u * b.abs())
            assert float(off.max()) <= e + 4 * u * math.log(v + 1)
        # ln z, and the mean octaves with z's error and its own
        assert float((entropy.double() - want[1]).abs().max()) <= (3 * e + 2.0 ** -20) * (1 + math.log(v + 1))
    assert kda().read_device_status() == 0
