"""What paged attention's operands keep of weights and queries, at sizes that show a lost bit."""
import numpy as np
import pytest
import torch

from tests import paged_reference as ref
from tests.test_gpu_paged import DEV, E4M3, ROWS, attend, attend_case, check_attend, i32, kda

pytestmark = pytest.mark.gpu


# The heavy key has weight 1 and 64K others 2^-a each: a between the powers of two, which e4m3
# holds exactly, and from 11 bits' reach to the floor of the split weights.
@pytest.mark.parametrize("heads,kv,run", ROWS)
@pytest.mark.parametrize("requests", [304, 1])  # whole units to a block; one cut into many shares
def test_a_heavy_first_key_and_a_long_tail_of_light_ones(heads, kv, run, requests):
    """The bound.  A light weight w is rounded to 11 bits, and where the split weights end, within
    2^-25 of the largest with errors that cancel over the 128 keys of a tile: within 2^-11 w + 2^-29
    on average.  The output's own rounding is up to 2^-8 (bf16 has 8 significant bits); 2^-13 for
    scores, sums and exponentials in fp32 (sums of 512 tiles: 2^-15)."""
    bs, n = 64, 1 << 16
    ctx = n + run
    kc, vc = torch.zeros(2, 1, bs, 128), torch.ones(2, 1, bs, 128)
    kc[0, 0, 0, 0] = 112.0
    vc[0, 0, 0, 0], vc[0, 0, 0, 1:64], vc[0, 0, 0, 64:] = 0.0, -1.0, 1.0
    vc[:, :, :, 100:] = 0.0  # the heavy key's value alone
    vc[0, 0, 0, 100:] = 1.0
    q = torch.zeros(requests * run, heads, 128, dtype=torch.bfloat16)
    q[:, :, 0] = 1.0
    one = torch.ones(2, 1, device=DEV)
    table = torch.ones(requests, -(-ctx // bs), dtype=torch.int32, device=DEV)
    table[:, 0] = 0
    for a in (10.6, 13.6, 15.2, 16.9, 19.4, 21.7):
        sm = float(np.float32(a * np.log(2.0) / 112.0))
        out = kda().paged_attention(q.to(DEV), i32(list(range(0, requests * run + 1, run))), table,
                                    i32([ctx] * requests), kc.to(E4M3).to(DEV), vc.to(E4M3).to(DEV), one,
                                    one, run, sm_scale=sm).double().cpu().view(requests, run, heads, 128)
        w = np.exp(-112.0 * sm)
        keys = (n + torch.arange(run, dtype=torch.float64)).view(1, run, 1, 1)  # light keys of a row
        heavy, light = vc[0, 0, 0].double(), vc[1, 0, 0].double()
        want = (heavy + keys * w * light) / (1 + keys * w)
        mean = (heavy.abs() + keys * w * light.abs()) / (1 + keys * w)
        bound = want.abs() * 2.0 ** -8 + mean * (2.0 ** -11 + 2.0 ** -13) + keys * 2.0 ** -29 / (1 + keys * w)
        worst = ((out - want).abs() / bound).max().item()
        assert worst <= 1, (a, worst)
    assert kda().read_device_status() == 0


@pytest.mark.parametrize("heads,kv,run", ROWS)
def test_queries_of_one_tile_that_differ_in_size(heads, kv, run):
    """A row's result does not depend on the size of the rows that share its tile: rows 2^34 apart,
    each within the bound of its own scores."""
    c = attend_case(run, [run, 1], [700, 300], heads, kv, 32)
    rows = c["q"].shape[0] * heads
    power = torch.linspace(-10, 24, rows).round()[torch.randperm(rows, generator=torch.Generator().manual_seed(run))]
    c["q"] = (c["q"].float() * torch.exp2(power).view(-1, heads, 1)).to(torch.bfloat16)
    check_attend(c)


@pytest.mark.parametrize("heads,kv,run", ROWS)
@pytest.mark.parametrize("size", [1e4, 1e9, 1e30])
def test_a_huge_finite_query_stays_in_its_row(heads, kv, run, size):
    c = attend_case(run, [run], [333], heads, kv, 64)
    c["q"][0, 1] *= size
    check_attend(c)


@pytest.mark.parametrize("heads,kv,run", ROWS)
@pytest.mark.parametrize("power", [-6, -9, -12])
def test_small_elements_of_a_query_are_exact(heads, kv, run, power):
    """All but one element of a query 2^-6 to 2^-13 of its largest, which meets zeros: the scores are
    the small elements' alone, and their rounding would show."""
    c = attend_case(run, [run, 1], [500, 300], heads, kv, 32, spoil=False)
    g = torch.Generator().manual_seed(run)
    size = torch.exp2(power - torch.rand(c["q"].shape, generator=g)) * 2.0 ** 7
    c["q"] = torch.where(c["q"] < 0, -size, size).to(torch.bfloat16)
    c["q"][:, :, 0] = 2.0 ** 7
    c["kc"].view(torch.uint8)[..., 0] = 0
    check_attend(c, sm_scale=2.0 ** (-9 - power))


@pytest.mark.parametrize("heads,kv,run", ROWS)
def test_elements_far_below_a_querys_largest(heads, kv, run):
    """Elements below 2^-13 of the largest, which meets zeros, are held within 2^-21 of it: a score is
    off by that times the sum of |k|, and a weight and the sum by as much each."""
    c = attend_case(run, [run], [260], heads, kv, 32, spoil=False)
    g = torch.Generator().manual_seed(run)
    c["q"] = (torch.randn(c["q"].shape, generator=g) * 2.0 ** -8).to(torch.bfloat16)
    c["q"][:, :, 0] = 2.0 ** 7
    c["kc"].view(torch.uint8)[..., 0] = 0
    out = attend(c, sm_scale=1.0).double().cpu().numpy()
    o, spread, top, most = ref.attention(c["q"], c["cu"], c["tables"], c["ctx"], c["kc"], c["vc"], c["ks"],
                                         c["vs"], sm_scale=1.0)
    k = (c["kc"].float().abs().sum(-1) * c["ks"][..., None]).max().item()
    off = np.expm1(2 * 2.0 ** 7 * 2.0 ** -21 * k)
    assert off < 0.1
    bound = 2.0 ** -8 * np.abs(o) + (2.0 ** -9 + 2.0 ** -16 * top + off) * spread + 2.0 ** -25 * most
    assert (np.abs(out - o) <= bound).all()
    assert kda().read_device_status() == 0


@pytest.mark.parametrize("heads,kv,run", ROWS)
@pytest.mark.parametrize("power", [-110, 0, 107])
def test_queries_near_the_ends_of_the_range(heads, kv, run, power):
    """Elements 2^power and 1.25 2^(power - 1) keep their order: the first meets a key of 1, the second
    one of 1.5, so the first key has the larger score, by far where sm_scale undoes the power."""
    c = attend_case(run, [run], [run + 2], heads, kv, 16, spoil=False)
    c["q"][:] = 0
    c["q"][:, :, 0], c["q"][:, :, 1] = 2.0 ** power, 1.25 * 2.0 ** (power - 1)
    kc = torch.zeros(c["kc"].shape)
    page = c["tables"][0][0]
    kc[page, :, 0, 0], kc[page, :, 1, 1] = 1.0, 1.5
    c["kc"], c["ks"] = kc.to(E4M3), torch.full_like(c["ks"], 2.0 ** min(-power, 100))
    check_attend(c, sm_scale=4.0)


@pytest.mark.parametrize("heads,kv,run", ROWS)
@pytest.mark.parametrize("where", ["first", "middle", "last", "alternate"])
def test_pages_of_zero_values_keep_their_keys_weights(heads, kv, run, where):
    """A page of zeros has the smallest scale that an append gives, 2^-100.  Its keys take their part of
    the sum whether they come before, between or after pages of values."""
    c = attend_case(run, [run, run], [5000, 700], heads, kv, 64, q_size=0.3)
    for table, ctx in zip(c["tables"], c["ctx"]):
        n = -(-ctx // 64)
        zero = dict(first=range(n // 2), middle=range(n // 4, n - n // 4), last=range(n // 2, n),
                    alternate=range(0, n, 2))[where]
        for j in zero:
            c["vc"].view(torch.uint8)[table[j]] = 0
            c["vs"][table[j]] = 2.0 ** -100
    check_attend(c)
