"""The vocabulary calls at the ends of their sizes, and from two host threads at once."""
import math
import threading

import pytest
import torch

from tests import vocab_bounds as bounds
from tests.test_gpu_vocab import BF16, DEV, F32, calls, kda, same

MOST = 2 ** 30


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,shift,v", [(BF16, 0, MOST), (BF16, 5, MOST - 3), (F32, 0, MOST), (F32, 3, MOST - 1)])
def test_logprobs_of_the_largest_vocabularies(dtype, shift, v):
    """Few values, so that sums are known: weights of 2^-13 and, in known places, larger entries."""
    x = torch.full((v + shift,), -10.0, dtype=dtype, device=DEV)[shift:].view(1, v)
    at = torch.tensor([0, 1, 7, 2 ** 24 + 1, v // 2, v - 9, v - 2, v - 1], device=DEV)
    x[0, at] = torch.tensor([1.0, -1.0, 0.5, 3.0, 3.0, 2.0, -2.0, 2.5], dtype=dtype, device=DEV)
    scale = torch.tensor([math.log(2.0)], device=DEV)
    s = float(scale.double())
    got = kda().token_logprobs(x, torch.tensor([v - 1], dtype=torch.int32, device=DEV), top_k=12, inv_temperature=scale)
    lp, entropy, ids, best = (a.cpu().double() for a in got)
    order = [2 ** 24 + 1, v // 2, v - 1, v - 9, 0, 7, 1, v - 2, 2, 3, 4, 5]
    assert ids[0].tolist() == order
    top = torch.tensor([3.0, 3.0, 2.5, 2.0, 1.0, 0.5, -1.0, -2.0, -10.0, -10.0, -10.0, -10.0], dtype=torch.float64)
    e, many = ((top[:8] - 3) * s).exp(), math.exp(-13 * s)
    z = float(e.sum()) + (v - 8) * many
    # a row is eight CTAs'; a weight's own error is 3 u 13 octaves and the exponential's
    error = bounds.U * (v / (8 * 512) + 64 + 40) + 2.0 ** -22
    want = (top - 3) * s - math.log(z)
    assert float((best[0] - want).abs().max()) <= error + 8 * bounds.U * math.log(v)
    assert abs(float(lp[0]) - float(want[2])) <= error + 8 * bounds.U * math.log(v)
    mean = (float((e * (top[:8] - 3) * s).sum()) + (v - 8) * many * -13 * s) / z
    assert abs(float(entropy[0]) - (math.log(z) - mean)) <= (3 * error + 2.0 ** -20) * (1 + math.log(v))
    assert kda().read_device_status() == 0


@pytest.mark.gpu
def test_hundreds_of_thousands_of_short_rows():
    t, v = 200_003, 5
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(t, v, generator=g, device=DEV)
    tokens = torch.randint(-1, v, (t,), generator=g, device=DEV, dtype=torch.int32)
    lp, entropy, ids, best = kda().token_logprobs(x, tokens, top_k=2)
    logq = torch.log_softmax(x.double(), 1)
    off = tokens < 0
    # a weight is within 2^-22 and three roundings of its (at most 12) octaves; logarithms and differences
    error = 2.0 ** -21 + 64 * bounds.U
    want = logq.gather(1, tokens.clamp(min=0).long()[:, None])[:, 0].masked_fill(off, 0)
    assert float(((lp - want).abs() - 4 * bounds.U * want.abs()).max()) <= error
    order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :2]
    assert torch.equal(ids, torch.where(off[:, None], -1, order).int())
    live = ~off
    assert float((best - logq.gather(1, order))[live].abs().max()) <= error + 4 * bounds.U * 20
    assert float((entropy - (-logq.exp() * logq).sum(1))[live].abs().max()) <= 4 * error
    at = torch.stack([torch.randint(0, v, (t,), generator=g, device=DEV), torch.full((t,), -1, device=DEV)], 1).int()
    val = torch.log(torch.rand(t, 2, generator=g, device=DEV) * 0.9 + 0.05)
    w = torch.rand(t, generator=g, device=DEV) + 0.5
    want = bounds.distill(x, at, val, 1.0, True)
    loss, d = kda().distill_topk_grad(x, at, val, w, tail=True)
    assert float(((loss - want["loss"]).abs() - want["loss_error"]).max()) <= 0
    grad = want["grad"] * w[:, None]
    limit = want["grad_error"] * w[:, None] * (1 + bounds.U) + bounds.U * grad.abs() + 2.0 ** -133
    assert float(((d - grad).abs() - limit).max()) <= 0
    assert kda().read_device_status() == 0


@pytest.mark.gpu
def test_calls_from_two_host_threads():
    runs = [calls(70), calls(71, t=150, v=9001)]
    wants = [run() for run in runs]
    torch.cuda.synchronize()
    gots, failed = [[], []], []

    def loop(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(40):
                    gots[i].append(runs[i]())
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # pragma: no cover
            failed.append(e)

    threads = [threading.Thread(target=loop, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    assert all(same(got, want) for want, some in zip(wants, gots) for got in some) and len(gots[0]) == len(gots[1]) == 40
