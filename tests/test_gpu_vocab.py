"""Log probabilities and distillation over vocabulary rows against plain implementations in 64 bits."""
import math

import pytest
import torch

from tests import vocab_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
INVALID = -1
INF = math.inf


def kda():
    import kimi_delta_attention_03_gb300 as m
    return m


def gen(seed):
    return torch.Generator().manual_seed(seed)


def logits(seed, t, v, dtype, spread=2.5):
    g = gen(seed)
    x = torch.randn(t, v, generator=g) * spread
    x[torch.arange(t), torch.randint(0, v, (t,), generator=g)] += 8 * torch.rand(t, generator=g)
    return x.to(dtype)


def strided(x, pad, shift):
    """x on the GPU, in rows `pad` elements wider, `shift` elements behind an aligned address."""
    t, v = x.shape
    wide = torch.full((t * (v + pad) + shift + 8,), 7.0, dtype=x.dtype, device=DEV)
    y = wide[shift:shift + t * (v + pad)].view(t, v + pad)[:, :v]
    y.copy_(x)
    return y


# --------------------------------------------------------------------------------- log probabilities
def check_logprobs(x, tokens=None, k=0, scale=None, on_gpu=None):
    """The rows' values are finite or -inf, and some entry is finite."""
    want = ref.logprobs(x, tokens, k, scale)
    got = kda().token_logprobs(on_gpu if on_gpu is not None else x.to(DEV),
                               None if tokens is None else tokens.to(DEV), top_k=k,
                               inv_temperature=None if scale is None else scale.to(DEV))
    got = [None if a is None else a.cpu() for a in got]
    v = x.shape[1]
    e = ref.sum_error(v)
    s = torch.ones(len(x)) if scale is None else scale
    # y - lse: two roundings of y and one of the result, the logarithm's own
    for a, b in ((got[0], want[0]), (got[3], want[3])):
        if a is None or not a.numel():
            continue
        assert a.dtype is F32 and torch.equal(a == -INF, b == -INF)
        fine = b > -INF
        off = (a.double() - b)[fine].abs() - 4 * ref.U * b[fine].abs()
        assert float(off.max() if off.numel() else 0) <= e + 4 * ref.U * math.log(v + 1) + 1e-9
    # entropy: ln z and the mean octaves, at most ln V each, the second to 2 e and what weights lose
    assert float((got[1].double() - want[1]).abs().max()) <= (3 * e + 2.0 ** -20) * (1 + math.log(v + 1))
    assert torch.equal(got[2], want[2])
    assert s.numel() == len(x)
    assert kda().read_device_status() == 0
    return got


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("v", [1, 2, 7, 8, 9, 31, 500, 4095, 8192, 8209, 50001, 131075])
@pytest.mark.parametrize("k", [0, 1, 5, 128])
def test_logprobs(dtype, v, k):
    x = logits(v + k, 5, v, dtype)
    tokens = torch.randint(0, v, (5,), generator=gen(v), dtype=torch.int32)
    check_logprobs(x, tokens, k)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("t,v", [(1, 32000), (29, 9001), (58, 20011), (115, 33000), (230, 5003), (700, 700)])
def test_logprobs_cluster_sizes_and_temperatures(dtype, t, v):
    x = logits(t, t, v, dtype)
    scale = 0.3 + 2 * torch.rand(t, generator=gen(t))
    tokens = torch.randint(-2, v, (t,), generator=gen(t + 1), dtype=torch.int32).clamp(min=-1)
    check_logprobs(x, tokens, 20, scale)


@pytest.mark.parametrize("dtype,shifts", [(BF16, range(8)), (F32, range(4))])
def test_logprobs_rows_at_any_address_and_stride(dtype, shifts):
    for shift in shifts:
        for v in (3, 17, 1003, 40003):
            x = logits(shift, 4, v, dtype)
            check_logprobs(x, None, 6, on_gpu=strided(x, (5 * shift + v) % 13, shift))


@pytest.mark.parametrize("t,v", [(230, 300007), (1, 2500003)])
def test_logprobs_vocabularies_with_shared_batch_maxima(t, v):
    """Vocabularies of which a thread reads more batches than it keeps maxima."""
    g = torch.Generator(device=DEV).manual_seed(t)
    x = (torch.randn(t, v, generator=g, device=DEV) * 2).to(BF16)
    _, entropy, ids, best = kda().token_logprobs(x, top_k=50)
    for i in range(0, t, 60):
        want = ref.logprobs(x[i:i + 1].cpu(), None, 50)
        assert torch.equal(ids[i:i + 1].cpu(), want[2])
        assert float((best[i].cpu() - want[3][0]).abs().max()) <= 2 * ref.sum_error(v)
        assert float((entropy[i].cpu() - want[1][0]).abs()) <= 4 * ref.sum_error(v) * math.log(v)
    assert kda().read_device_status() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("v", [40, 3001, 70001])
def test_logprobs_equal_and_sorted_entries(dtype, v):
    """Ties go to the lowest index, zeros of both signs are equal, and orders that make every entry a
    candidate end."""
    g = gen(v)
    ramp = torch.linspace(-9, 9, v)
    x = torch.stack([
        torch.full((v,), 1.5), torch.zeros(v), ramp, ramp.flip(0),
        torch.where(torch.arange(v) % 2 == 0, -0.0, 0.0),
        torch.randint(0, 3, (v,), generator=g).float(),
        torch.where(torch.arange(v) >= v - 30, 4.0, -4.0),
        ramp.abs(), torch.randn(v, generator=g).round(),
    ]).to(dtype)
    for k in (1, 20, 128):
        check_logprobs(x, None, k)
        check_logprobs(x.repeat(60 if v > 9000 else 70, 1), None, k)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("t,v", [(6, 131072), (6, 131069), (330, 40007), (6, 700001)])
def test_logprobs_equal_entries_by_the_thousand(dtype, t, v):
    """Fewer tokens than alternatives beside a mask's value, and rows of few values: of the equal entries the
    first ones, wherever they are."""
    g = gen(v)
    low = torch.finfo(dtype).min
    x = torch.full((6, v), low)
    x[0, torch.randint(0, v, (4,), generator=g)] = torch.randn(4, generator=g)
    x[1] = -1.5
    x[1, v - 3:] = 2.0
    x[2] = torch.where(torch.arange(v) < v // 2, -7.0, 0.1)
    x[3] = 0.1
    x[3, ::7] = -0.3
    x[4, v // 2:] = torch.randint(0, 2, (v - v // 2,), generator=g).float()
    x[5, 9000:] = 3.0
    x = x.to(dtype).repeat(t // 6, 1)
    for k in (3, 20, 128):
        check_logprobs(x, None, k)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_logprobs_masks(dtype):
    """Rows held to a few tokens, by -inf and by the type's lowest value, and rows all of that value."""
    v, low = 5003, torch.finfo(dtype).min
    g = gen(3)
    x = logits(3, 12, v, dtype)
    keep = torch.zeros(12, v, dtype=torch.bool)
    keep.scatter_(1, torch.randint(0, v, (12, 3), generator=g), True)
    x[:4] = torch.where(keep[:4], x[:4], -INF)
    x[4:8] = torch.where(keep[4:8], x[4:8], low)
    x[8] = low
    x[9, :] = -INF
    x[9, v - 1] = low
    x[10, :v // 2] = -INF
    x[11, 1:] = -INF
    tokens = x.float().argmax(1).to(torch.int32)
    check_logprobs(x, tokens, 8)
    check_logprobs(x.repeat(60, 1), tokens.repeat(60), 8)
    tokens = torch.tensor([int((~keep[i]).nonzero()[0]) for i in range(12)], dtype=torch.int32)
    got = check_logprobs(x, tokens, 3)
    assert torch.equal(got[0][:4], torch.full((4,), -INF))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("t", [4, 400])
def test_logprobs_rows_without_a_distribution(dtype, t):
    v = 9001
    x = logits(5, t, v, dtype)
    x[0] = -INF
    x[1, v - 1] = math.nan
    x[2, 17] = INF
    tokens = torch.full((t,), 17, dtype=torch.int32)
    lp, entropy, ids, best = kda().token_logprobs(x.to(DEV), tokens.to(DEV), top_k=4)
    for a in (lp, entropy, best):
        assert a[:3].isnan().all() and a[3:].isfinite().all()
    assert (ids[:3] == -1).all()
    want = ref.logprobs(x[3:], tokens[3:], 4)
    assert torch.equal(ids[3:].cpu(), want[2])
    scale = torch.tensor([0.0, -1.0, math.nan, INF] + [1.0] * (t - 4))
    lp, entropy, ids, best = kda().token_logprobs(logits(6, t, v, dtype).to(DEV), tokens.to(DEV), top_k=4,
                                                  inv_temperature=scale.to(DEV))
    for a in (lp, entropy, best):
        assert a[:4].isnan().all() and a[4:].isfinite().all()
    assert (ids[:4] == -1).all()
    assert kda().read_device_status() == 0


def test_logprobs_large_values_and_steep_temperatures():
    v = 4001
    x = logits(7, 6, v, F32)
    x[0] += 1e4
    x[1] *= 1e30
    x[2] *= 1e-30
    x[3] = torch.where(torch.arange(v) == 5, 3e38, -3e38)
    scale = torch.tensor([1.0, 1.0, 1.0, 1.0, 1e6, 1e-6])
    want = ref.logprobs(x, x.argmax(1).to(torch.int32), 3, scale)
    got = kda().token_logprobs(x.to(DEV), x.argmax(1).to(torch.int32).to(DEV), top_k=3,
                               inv_temperature=scale.to(DEV))
    for a, b in ((got[0], want[0]), (got[3], want[3])):
        # differences of the logits are exact here or rounded once
        fine = b.abs() < 1e38
        assert float(((a.cpu().double() - b).abs() - 2.0 ** -21 * b.abs())[fine].max()) <= ref.sum_error(v)
        assert (a.cpu()[~fine] <= -9e37).all()
    assert float((got[1].cpu() - want[1]).abs().max()) <= 20 * ref.sum_error(v)
    assert torch.equal(got[2].cpu(), want[2])


def test_logprobs_token_outside_the_vocabulary():
    x = logits(8, 3, 100, F32)
    tokens = torch.tensor([5, 100, 7], dtype=torch.int32)
    got = kda().token_logprobs(x.to(DEV), tokens.to(DEV), top_k=2)
    assert kda().read_device_status() == INVALID
    want = ref.logprobs(x, torch.tensor([5, -1, 7], dtype=torch.int32), 2)
    assert torch.equal(got[2].cpu(), want[2]) and float(got[0][1]) == 0 and float(got[1][1]) == 0
    assert torch.equal(got[3].cpu() == -INF, want[3] == -INF)


# -------------------------------------------------------------------------------------- distillation
def teacher(seed, x, k, tail, absent=0.0, empty=0.0):
    """Entries of a teacher near x: its k largest."""
    g = gen(seed)
    t, v = x.shape
    z = x.double().nan_to_num(0, 30, -30).clamp(-30, 30) + 0.8 * torch.randn(t, v, generator=g)
    val, ids = torch.topk(z, k, dim=1)
    if tail:
        val = val - torch.logsumexp(z, 1, keepdim=True)
    ids = ids.to(torch.int32)
    ids[(torch.rand(t, k, generator=g) < absent) | (torch.rand(t, 1, generator=g) < empty)] = -1
    return ids, val.float()


def near(got, want, error):
    got, want = got.double().cpu(), want.double()
    assert torch.equal(got.isinf(), want.isinf()) and not got.isnan().any()
    off = torch.where(want.isinf(), 0.0, (got - want).abs() - error)
    assert float(off.max()) <= 0, float(off.max())


def check_distill(x, ids, val, scale=1.0, tail=False, on_gpu=None, weight=None, out=None):
    t, v = x.shape
    want = ref.distill(x, ids, val, scale, tail)
    y = x.to(DEV) if on_gpu is None else on_gpu
    i, a = ids.to(DEV), val.to(DEV)
    loss, stats = kda().distill_topk(y, i, a, scale, tail)
    near(loss, want["loss"], want["loss_error"])
    read = want["stats"][:, 1] > 0
    assert torch.equal(stats[:, [0, 2]].cpu().double(), want["stats"][:, [0, 2]])
    e = ref.sum_error(v)
    near(stats[:, [1, 3]], want["stats"][:, [1, 3]], e * want["stats"][:, [1, 3]])
    assert (stats[~read] == 0).all()
    if weight is None:
        weight = 0.5 + torch.rand(t, generator=gen(t))
    w = weight.to(DEV)
    d = kda().distill_topk_bwd(w, y, i, a, stats, scale, tail, d_logits=out)
    w64 = weight.double()[:, None]
    half = ref.step(x.dtype)
    bound = want["grad_error"] * w64.abs() + half * (want["grad"] * w64).abs() * (1 + half) + 2.0 ** -133
    near(d, want["grad"] * w64, bound)
    d = d.clone()
    loss2, d2 = kda().distill_topk_grad(y, i, a, w, scale, tail, d_logits=out)
    near(loss2, want["loss"], want["loss_error"])  # (summed in another order than loss)
    near(d2, want["grad"] * w64, bound)
    assert kda().read_device_status() == 0
    return loss, d, d2


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("v,k", [(2, 1), (9, 3), (300, 256), (1000, 64), (8209, 1), (32000, 20), (50001, 64),
                                 (131077, 256)])
def test_distill(dtype, tail, v, k):
    x = logits(v, 4, v, dtype)
    ids, val = teacher(v + 1, x, k, tail, absent=0.1 if k > 3 else 0.0)
    check_distill(x, ids, val, 1.0, tail)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("t,v", [(1, 70000), (19, 40000), (38, 40001), (76, 33000), (160, 900), (640, 130)])
def test_distill_cluster_sizes_absent_entries_and_rows(dtype, t, v):
    x = logits(t, t, v, dtype)
    ids, val = teacher(t + 1, x, 12, True, absent=0.3, empty=0.2)
    check_distill(x, ids, val, 0.5, True)
    check_distill(x, ids, val * 3 - 5, 0.5, False)


def test_distill_many_large_rows():
    """More rows than L2 keeps at a time: each is several CTAs'.  Some against 64 bits, all against the
    two calls of one CTA a row."""
    t, v = 620, 90007
    g = torch.Generator(device=DEV).manual_seed(3)
    x = (torch.randn(t, v, generator=g, device=DEV) * 2).to(BF16)
    few = torch.arange(0, t, 103)
    ids, val = teacher(4, x[few].cpu(), 40, True, absent=0.1)
    at = torch.arange(t) % len(few)
    all_ids, all_val, w = ids[at].to(DEV), val[at].to(DEV), torch.rand(t, generator=gen(5)).to(DEV)
    loss, d = kda().distill_topk_grad(x, all_ids, all_val, w, tail=True)
    other, stats = kda().distill_topk(x, all_ids, all_val, tail=True)
    # both within the bound of 64 bits of the same value
    e = ref.sum_error(v)
    assert float((loss - other).abs().max()) <= 2 * (3 * e + 2.0 ** -20 * 200)
    alone = kda().distill_topk_bwd(w, x, all_ids, all_val, stats, tail=True)
    assert float(((d - alone).float().abs() - 2.0 ** -7 * alone.float().abs()).max()) <= 2.0 ** -16
    for k, i in enumerate(few.tolist()):
        j = int(at[i])
        want = ref.distill(x[i:i + 1].cpu(), ids[j:j + 1], val[j:j + 1], 1.0, True)
        near(loss[i:i + 1], want["loss"], want["loss_error"])
        weight = float(w[i])
        bound = want["grad_error"] * weight + 2.0 ** -8 * (want["grad"] * weight).abs() * (1 + 2.0 ** -8) + 2.0 ** -133
        near(d[i:i + 1], want["grad"] * weight, bound)
    assert kda().read_device_status() == 0


def test_distill_largest_rows():
    for v, dtype in ((393216, F32), (786432, BF16), (393215, F32), (786425, BF16)):
        x = logits(v, 2, v, dtype)
        ids, val = teacher(1, x, 30, True)
        check_distill(x, ids, val, 1.0, True)


def test_distill_teacher_that_names_every_token():
    x = logits(1, 3, 40, F32)
    ids, val = teacher(2, x, 40, False)
    check_distill(x, ids, val)
    ids, val = teacher(2, x, 39, True)
    check_distill(x, ids, val, 1.0, True)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tail", [False, True])
def test_distill_tokens_named_more_than_once(dtype, tail):
    x = logits(2, 6, 20011, dtype)
    ids, val = teacher(3, x, 24, tail)
    val -= 1.0 if tail else 0.0
    ids[0] = ids[0, 0]
    ids[1, 5:8] = ids[1, 4]
    ids[2, ::2] = ids[2, 1::2]
    ids[3, 20] = 20010
    ids[3, 3] = 20010
    ids[4] = 0
    first = check_distill(x, ids, val, 1.0, tail)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(first, check_distill(x, ids, val, 1.0, tail)))


@pytest.mark.parametrize("tail", [False, True])
def test_calls_on_short_rows_repeat_their_bits(tail):
    """Rows so short that a CTA's warps are far apart."""
    x = logits(30, 600, 300, BF16)
    ids, val = teacher(31, x, 200, tail, absent=0.2)
    x, ids, val, w = x.to(DEV), ids.to(DEV), val.to(DEV), torch.ones(600, device=DEV)

    def run():
        return [*kda().distill_topk(x, ids, val, 1.0, tail), *kda().distill_topk_grad(x, ids, val, w, 1.0, tail),
                *kda().token_logprobs(x, top_k=60)[1:]]
    want = run()
    for _ in range(30):
        assert all(torch.equal(a, b) for a, b in zip(run(), want))


@pytest.mark.parametrize("dtype,shifts", [(BF16, range(8)), (F32, range(4))])
def test_distill_rows_at_any_address_and_stride(dtype, shifts):
    """Nothing beside the rows of a strided gradient is written."""
    for shift in shifts:
        for v in (5, 17, 1003, 40003):
            x = logits(shift, 3, v, dtype)
            ids, val = teacher(shift + 1, x, min(4, v - 1), True)
            pad = (5 * shift + v) % 13
            for other in (shift, (shift + 3) % 8):
                out = strided(torch.zeros_like(x), pad + other % 5, other)
                check_distill(x, ids, val, 1.0, True, on_gpu=strided(x, pad, shift), out=out)
                whole = out._base if out._base is not None else out
                mask = torch.ones_like(whole, dtype=torch.bool)
                mask[other:other + 3 * out.stride(0)].view(3, -1)[:, :v] = False
                assert (whole[mask] == 7).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("v", [41, 60001])
def test_distill_gradient_in_place_of_the_logits(dtype, v):
    x = logits(4, 5, v, dtype)
    ids, val = teacher(5, x, 9, True)
    w = torch.rand(5, generator=gen(6)).to(DEV)
    y = x.to(DEV)
    stats = kda().distill_topk(y, ids.to(DEV), val.to(DEV), tail=True)[1]
    want = kda().distill_topk_bwd(w, y, ids.to(DEV), val.to(DEV), stats, tail=True)
    loss, both = kda().distill_topk_grad(y, ids.to(DEV), val.to(DEV), w, tail=True)
    a, b = x.to(DEV), x.to(DEV)
    assert kda().distill_topk_bwd(w, a, ids.to(DEV), val.to(DEV), stats, tail=True, d_logits=a) is a
    got = kda().distill_topk_grad(b, ids.to(DEV), val.to(DEV), w, tail=True, d_logits=b)
    assert torch.equal(a, want) and torch.equal(b, both) and torch.equal(got[0], loss)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_distill_masked_logits_and_weights_of_zero(dtype):
    v = 9001
    x = logits(7, 8, v, dtype)
    ids, val = teacher(8, x, 6, True)
    x[0, 100:] = -INF            # some entries' tokens, perhaps all, and most others
    x[1, ids[1].long()] = -INF   # every entry's token: infinite loss, finite gradient
    keep = torch.zeros(v, dtype=torch.bool)
    keep[ids[2].long()] = True
    x[2, ~keep] = -INF           # nothing but the entries' tokens: with r > 0 infinite
    x[3] = torch.where(keep, x[3], torch.finfo(dtype).min)
    x[4] = torch.finfo(dtype).min
    val[5] = -INF                # entries without probability
    val[6, :3] = -INF
    w = torch.tensor([1.0, 0.5, 1.0, 1.0, 1.0, 1.0, 1.0, 0.0])
    check_distill(x, ids, val, 1.0, True, weight=w)
    check_distill(x, ids, val, 1.0, False, weight=w)


@pytest.mark.parametrize("tail", [False, True])
def test_distill_values_beyond_log_probabilities(tail):
    """Entries whose probabilities sum to more than 1 leave nothing, values of absent entries do not matter, and a
    value that is NaN or +inf makes its row's loss NaN, no other's."""
    x = logits(42, 6, 3001, F32)
    ids, val = teacher(43, x, 9, True)
    val[0] += 2.0
    val[1, 0] = 12.0
    val[2, 3] = 0.0
    ids[3, 4:] = -1
    val[3, 4:] = math.nan
    val[4] = -40.0  # next to nothing: with tail all of it is left
    val[4, 0] = -3e38
    check_distill(x, ids, val.nan_to_num(0.0), 1.0, tail)
    want = kda().distill_topk_grad(x.to(DEV), ids.to(DEV), val.nan_to_num(0.0).to(DEV), torch.ones(6, device=DEV),
                                   tail=tail)
    got = kda().distill_topk_grad(x.to(DEV), ids.to(DEV), val.to(DEV), torch.ones(6, device=DEV), tail=tail)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    val[3, 4:] = 0.0
    for bad in (math.nan, math.inf):
        v = val.clone()
        v[5, 2] = bad
        loss, d = kda().distill_topk_grad(x.to(DEV), ids.to(DEV), v.to(DEV), torch.ones(6, device=DEV), tail=tail)
        assert torch.equal(loss[:5], want[0][:5]) and torch.equal(d[:5], want[1][:5])
        assert not loss[5].isfinite() and not d[5].isfinite().all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("scale", [1e-6, 30.0, 1e6])
def test_distill_extreme_scales_and_far_logits(dtype, scale):
    """Scales at which a row's maximum times the scale is far beyond what one fma holds, and logits far off."""
    x = logits(40, 6, 9001, F32, spread=1.0)
    x[1] += 3e4
    x[2] -= 3e4
    x[3] *= 2.0 ** 40
    x[4] = (x[4] * 64).round() / 64
    x = x.to(dtype)
    ids, val = teacher(41, x, 10, True)
    check_distill(x, ids, val, scale, True)
    check_distill(x, ids, val, scale, False)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_distill_rows_without_a_distribution(dtype):
    v = 30001
    x = logits(9, 5, v, dtype)
    ids, val = teacher(10, x, 6, True)
    x[0] = -INF
    x[1, 3] = math.nan
    x[2, int(ids[2, 0])] = INF
    ids[3] = -1
    loss, d = kda().distill_topk_grad(x.to(DEV), ids.to(DEV), val.to(DEV), torch.ones(5, device=DEV), tail=True)
    assert loss[:3].isnan().all() and loss[3] == 0 and loss[4].isfinite()
    assert d[:3].isnan().any(1).all() and (d[3] == 0).all() and d[4].isfinite().all()
    # weight 0: zeros whatever the logits are
    w = torch.tensor([0.0, 0.0, 0.0, 1.0, 1.0], device=DEV)
    loss, d = kda().distill_topk_grad(x.to(DEV), ids.to(DEV), val.to(DEV), w, tail=True)
    assert loss[:3].isnan().all() and (d[:4] == 0).all() and (d[4] != 0).any()
    # a row whose loss has no gradient is skipped
    loss, stats = kda().distill_topk(x.to(DEV), ids.to(DEV), val.to(DEV), tail=True)
    w = torch.tensor([0.0, 0.0, 0.0, 1.0, 1.0], device=DEV)
    d = kda().distill_topk_bwd(w, x.to(DEV), ids.to(DEV), val.to(DEV), stats, tail=True)
    assert (d[:4] == 0).all() and (d[4] != 0).any()
    assert kda().read_device_status() == 0


def test_distill_entry_outside_the_vocabulary_is_absent_and_reported():
    x = logits(11, 3, 500, F32)
    ids, val = teacher(12, x, 4, True)
    bad = ids.clone()
    bad[1, 2] = 500
    ids[1, 2] = -1
    want = kda().distill_topk_grad(x.to(DEV), ids.to(DEV), val.to(DEV), torch.ones(3, device=DEV), tail=True)
    assert kda().read_device_status() == 0
    got = kda().distill_topk_grad(x.to(DEV), bad.to(DEV), val.to(DEV), torch.ones(3, device=DEV), tail=True)
    assert kda().read_device_status() == INVALID
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("tail", [False, True])
def test_distill_gradient_against_differences(tail):
    """Central differences of the 64-bit loss, h = 1e-5: off by h^2 times a third derivative below 1 and
    2^-52 / h, so by 1e-9 at most, beside the kernel's own error."""
    v = 60
    x = logits(13, 3, v, F32, spread=1.0)
    ids, val = teacher(14, x, 5, tail)
    w = torch.tensor([1.0, 0.3, 2.0])
    _, d = kda().distill_topk_grad(x.to(DEV), ids.to(DEV), val.to(DEV), w.to(DEV), 0.7, tail)
    h = 1e-5
    up, down = x.double().repeat(v, 1, 1), x.double().repeat(v, 1, 1)
    for j in range(v):
        up[j, :, j] += h
        down[j, :, j] -= h
    flat = lambda a: ref.distill(a.reshape(-1, v), ids.repeat(v, 1), val.repeat(v, 1), 0.7, tail)["loss"]
    slope = ((flat(up) - flat(down)) / (2 * h)).view(v, 3).T * w.double()[:, None]
    bound = ref.distill(x, ids, val, 0.7, tail)["grad_error"] * w.double()[:, None]
    assert float(((d.cpu().double() - slope).abs() - bound).max()) <= 2e-8


# ------------------------------------------------------------------------------------------ together
def test_teacher_records_its_alternatives_and_the_student_learns_from_them():
    """What token_logprobs returns for the target is what distill_topk takes: the loss of a student
    with the target's own logits is zero, and a step along the gradient brings a student nearer."""
    t, v, k = 40, 20011, 32
    target, student = logits(15, t, v, BF16).to(DEV), logits(16, t, v, F32).to(DEV)
    _, _, ids, best = kda().token_logprobs(target, top_k=k)
    loss, _ = kda().distill_topk(target, ids, best, tail=True)
    # both sides' logarithms of z, and r's from what rounded log probabilities leave
    assert float(loss.abs().max()) <= 4 * ref.sum_error(v) + 2.0 ** -17
    w = torch.full((t,), 1.0, device=DEV)
    before, d = kda().distill_topk_grad(student, ids, best, w, tail=True)
    near(before, ref.distill(student.cpu(), ids.cpu(), best.cpu(), 1.0, True)["loss"],
         ref.distill(student.cpu(), ids.cpu(), best.cpu(), 1.0, True)["loss_error"])
    after, _ = kda().distill_topk(student - 0.1 * d, ids, best, tail=True)
    assert (after < before).all()


def test_verified_drafts_answer_with_log_probabilities():
    """Rejected places carry -1 and are not read: their log probability adds nothing to a run's sum."""
    v, runs = 5003, [4, 1, 6, 3]
    t, cu = sum(runs), [0, 4, 5, 11, 14]
    x = logits(17, t, v, F32).to(DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    p = torch.softmax(x, 1)
    tokens = torch.multinomial(p, 1, generator=g)[:, 0].roll(1).to(torch.int32)
    _, _, out = kda().verify_draft(p, tokens, torch.tensor(cu, dtype=torch.int32, device=DEV),
                                   torch.rand(t, device=DEV, generator=g),
                                   torch.empty(4, v, device=DEV).exponential_(generator=g))
    lp, entropy, ids, best = kda().token_logprobs(x, out, top_k=3)
    want = ref.logprobs(x.cpu(), out.cpu(), 3)
    assert torch.equal(ids.cpu(), want[2]) and (lp[out < 0] == 0).all()
    assert float((lp.cpu() - want[0]).abs().max()) <= 2 * ref.sum_error(v) + 2.0 ** -20


def test_draft_distillation_example(capsys):
    """It runs, and its gradient in the output layer is the formula's, differentiated in 64 bits."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "draft_distillation.py")
    spec = importlib.util.spec_from_file_location("draft_distillation", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    assert example.main(3).isfinite().all() and "step 2" in capsys.readouterr().out
    g = torch.Generator(device=DEV).manual_seed(2)
    hidden = torch.randn(12, 16, generator=g, device=DEV)
    head = torch.randn(16, 300, generator=g, device=DEV) * 0.3
    ids, best = example.record(torch.randn(12, 300, generator=g, device=DEV) * 2)
    w = torch.rand(12, generator=g, device=DEV)
    loss, d = example.gradient(hidden, head, ids, best, w)
    h64, w64 = hidden.double().cpu(), w.double().cpu()
    x = (hidden @ head).cpu()
    want = ref.distill(x, ids.cpu(), best.cpu(), 1.0, True)
    # the product adds 12 terms in fp32: 13 roundings of each
    error = want["grad_error"] + 13 * ref.U * want["grad"].abs()
    off = (d.double().cpu() - h64.T @ (want["grad"] * w64[:, None])).abs()
    assert (off <= h64.abs().T @ (error * w64[:, None]) + 1e-30).all()


def calls(seed, t=37, v=30011):
    x = logits(seed, t, v, BF16).to(DEV)
    ids, val = teacher(seed, x.cpu(), 20, True, absent=0.1, empty=0.1)
    ids, val = ids.to(DEV), val.to(DEV)
    tokens = torch.randint(-1, v, (t,), generator=gen(seed), dtype=torch.int32).to(DEV)
    w = torch.rand(t, generator=gen(seed)).to(DEV)
    scale = (0.5 + torch.rand(t, generator=gen(seed))).to(DEV)

    def run(**kw):
        a = kda().token_logprobs(x, tokens, top_k=20, inv_temperature=scale, **kw)
        b = kda().distill_topk(x, ids, val, 0.5, True, **kw)
        c = kda().distill_topk_bwd(w, x, ids, val, b[1], 0.5, True, **kw)
        d = kda().distill_topk_grad(x, ids, val, w, 0.5, True, **kw)
        return [*a, *b, c, *d]
    return run


def same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


def test_calls_on_another_stream_give_the_same_bits():
    run = calls(20)
    want = run()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [run(stream=side) for _ in range(20)]
    torch.cuda.synchronize()
    assert all(same(g, want) for g in got)


def test_calls_captured_in_a_graph_and_replayed():
    run = calls(21)
    want = run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(3):
        for g in got:
            g.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(got, want)


def test_two_graphs_of_the_calls_replayed_at_once():
    runs = [calls(23), calls(24, t=90, v=50001)]
    wants = [run() for run in runs]
    torch.cuda.synchronize()
    graphs, gots, sides = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for run in runs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            gots.append(run())
    for _ in range(10):
        for g, side in zip(graphs, sides):
            with torch.cuda.stream(side):
                g.replay()
    torch.cuda.synchronize()
    assert all(same(got, want) for got, want in zip(gots, wants))


def test_calls_without_rows():
    x = torch.empty(0, 100, device=DEV)
    none = torch.empty(0, 3, dtype=torch.int32, device=DEV)
    val = torch.empty(0, 3, device=DEV)
    lp, entropy, ids, best = kda().token_logprobs(x, torch.empty(0, dtype=torch.int32, device=DEV), top_k=3)
    assert lp.shape == entropy.shape == (0,) and ids.shape == best.shape == (0, 3)
    loss, stats = kda().distill_topk(x, none, val)
    assert kda().distill_topk_bwd(loss, x, none, val, stats).shape == (0, 100)
    assert kda().distill_topk_grad(x, none, val, loss)[1].shape == (0, 100)


def test_rows_beyond_four_gigabytes():
    """Offsets of the last rows pass 32 bits of elements."""
    t, v = 40, 131072
    base = torch.empty(17000, v * 2, dtype=BF16, device=DEV)
    x = base[::436, :v][:t - 1]
    src = logits(22, x.shape[0], v, BF16)
    x.copy_(src)
    assert x.stride(0) * (x.shape[0] - 1) > 2 ** 31
    tokens = torch.arange(x.shape[0], dtype=torch.int32)
    check_logprobs(src[-3:], tokens[-3:], 5, on_gpu=x[-3:])
    got = kda().token_logprobs(x, tokens.to(DEV), top_k=5)
    want = kda().token_logprobs(src.to(DEV), tokens.to(DEV), top_k=5)
    assert same(got, want)
    ids, val = teacher(23, src, 8, True)
    w = torch.ones(x.shape[0], device=DEV)
    want = kda().distill_topk_grad(src.to(DEV), ids.to(DEV), val.to(DEV), w, tail=True)
    got = kda().distill_topk_grad(x, ids.to(DEV), val.to(DEV), w, tail=True, d_logits=x)
    assert torch.equal(got[0], want[0]) and torch.equal(x, want[1])


def test_python_checks():
    x = torch.zeros(3, 10, device=DEV)
    i = torch.zeros(3, dtype=torch.int32, device=DEV)
    ids, val = torch.zeros(3, 2, dtype=torch.int32, device=DEV), torch.zeros(3, 2, device=DEV)
    w = torch.zeros(3, device=DEV)
    m = kda()
    for bad in (lambda: m.token_logprobs(x.cpu()), lambda: m.token_logprobs(x.half()),
                lambda: m.token_logprobs(x.T), lambda: m.token_logprobs(x[0]),
                lambda: m.token_logprobs(x, i.long()), lambda: m.token_logprobs(x, i[:2]),
                lambda: m.token_logprobs(x, i.cpu()), lambda: m.token_logprobs(x, top_k=129),
                lambda: m.token_logprobs(x, top_k=-1), lambda: m.token_logprobs(x, inv_temperature=w.double()),
                lambda: m.distill_topk(x, ids[:2], val), lambda: m.distill_topk(x, ids, val.half()),
                lambda: m.distill_topk(x, ids[0], val), lambda: m.distill_topk(x, ids, val[:, :1]),
                lambda: m.distill_topk_bwd(w, x, ids, val, val), lambda: m.distill_topk_bwd(w[:2], x, ids, val, x),
                lambda: m.distill_topk_grad(x, ids, val, w, d_logits=x.bfloat16()),
                lambda: m.distill_topk_grad(x, ids, val, w, d_logits=x[:2])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: m.distill_topk(x, ids, val, 0.0), lambda: m.distill_topk(x, ids, val, math.nan),
                lambda: m.distill_topk(x[:, :2], ids, val, tail=True),
                lambda: m.distill_topk(x, torch.zeros(3, 0, dtype=torch.int32, device=DEV), val[:, :0]),
                lambda: m.distill_topk(x, torch.zeros(3, 257, dtype=torch.int32, device=DEV),
                                       torch.zeros(3, 257, device=DEV))):
        with pytest.raises(m.KdaError):
            bad()
