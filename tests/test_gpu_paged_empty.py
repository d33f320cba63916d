"""Units without keys: requests whose context is empty or shorter than their run."""
import random

import pytest
import torch

from tests.test_gpu_paged import ROWS, attend, attend_case, check_attend

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,kv,run", ROWS)
def test_many_units_without_keys_between_others(heads, kv, run):
    """Stretches of up to hundreds of units without a tile, which only order the warps of a block by
    their hand-overs, between units of one to eight tiles."""
    r = random.Random(run)
    runs, ctx = [], []
    while len(runs) < 2500:
        empty = r.choice([1, 2, 3, 7, 40, 300])
        runs += [r.choice([1, run]) for _ in range(empty)]
        ctx += [0] * empty
        for _ in range(r.randint(1, 2)):
            runs.append(r.choice([1, run, run]))
            ctx.append(r.choice([max(runs[-1] - 1, 0), runs[-1], 129 + run, 600, 1000]))
    runs[0] = run
    c = attend_case(run, runs, ctx, heads, kv, 64)
    out = check_attend(c)
    for a, b, k in zip(c["cu"], c["cu"][1:], ctx):
        if k == 0:
            assert (out[a:b] == 0).all()


@pytest.mark.parametrize("heads,kv,run", ROWS)
def test_nothing_but_units_without_keys(heads, kv, run):
    n = 3000
    c = attend_case(run, [run] * n, [0] * n, heads, kv, 16)
    assert torch.equal(check_attend(c), torch.zeros(n * run, heads, 128, dtype=torch.bfloat16, device="cuda"))


@pytest.mark.parametrize("heads,kv,run", ROWS)
def test_a_nan_value_does_not_reach_units_without_keys(heads, kv, run):
    """Segments share the place where a tile notes its first NaN value."""
    n = 1200
    ctx = [run + 40 if i % 3 == 0 else 0 for i in range(n)]
    c = attend_case(run, [run] * n, ctx, heads, kv, 16, spoil=False)
    raw = c["vc"].view(torch.uint8)
    for i in range(0, n, 3):
        raw[c["tables"][i][(ctx[i] - 1) // 16], :, (ctx[i] - 1) % 16, 5] = 0x7F  # the last token's value
    out = attend(c).view(n, run, heads, 128)
    empty = torch.tensor([k == 0 for k in ctx], device="cuda")
    assert (out[empty] == 0).all()
    seen = torch.zeros_like(out[~empty], dtype=torch.bool)
    seen[:, -1, :, 5] = True
    assert torch.equal(out[~empty].isnan(), seen)
