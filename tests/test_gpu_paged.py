"""The paged serving operators against plain host implementations in 64 bits."""
import random

import numpy as np
import pytest
import torch

from tests import paged_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
E4M3 = torch.float8_e4m3fn
INVALID = -1


def kda():
    import kimi_delta_attention_03_gb300 as m
    return m


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def cu_of(runs):
    return [0] + list(np.cumsum(runs))


# ------------------------------------------------------------------------------------------ plan
def plan_case(seed, n, run_hi, bs, ctx_hi, release=0.0, short=False, width_cut=0):
    r = random.Random(seed)
    runs = [r.randint(0, run_hi) for _ in range(n)]
    cached = [r.choice([0, 1, bs - 1, bs, bs + 1, r.randint(0, ctx_hi)]) for _ in range(n)]
    held = [-(-c // bs) + r.choice([0, 0, 0, 1, 2]) for c in cached]
    gone = [1 if r.random() < release else 0 for _ in range(n)]
    width = max([-(-(c + k) // bs) for c, k in zip(cached, runs)] + held) + 1 - width_cut
    width = max(width, max(held))
    need = sum(max(0, -(-(c + k) // bs) - h) for c, k, h in zip(cached, runs, held))
    spare = need // 2 if short else need + 3
    pages = list(range(sum(held) + spare))
    r.shuffle(pages)
    tables = [[-7] * width for _ in range(n)]
    for i in range(n):
        for j in range(held[i]):
            tables[i][j] = pages.pop()
    free = pages + [-9] * (sum(held) + 2)
    return dict(cached=cached, cu=cu_of(runs), tables=tables, held=held, free=free,
                count=len(pages), bs=bs, t=sum(runs), release=gone if release else None)


def run_plan(c, **kw):
    tables, free = i32(c["tables"]), i32(c["free"])
    got = kda().paged_plan(i32(c["cached"]), i32(c["cu"]), tables, i32(c["held"]), free,
                           i32([c["count"]]), c["bs"], c["t"],
                           release=None if c["release"] is None else i32(c["release"]), **kw)
    return [x.tolist() for x in got] + [tables.tolist(), free.tolist()]


def check_plan(c):
    want = ref.plan(c["cached"], c["cu"], c["tables"], c["held"], c["free"], c["count"], c["bs"],
                    c["t"], c["release"])
    got = run_plan(c)
    got[2] = got[2][0]
    for name, g, w in zip(("context", "held", "free_count", "positions", "slots", "tables", "free"),
                          got, want):
        assert g == w, name
    assert kda().read_device_status() == 0


@pytest.mark.parametrize("n,run_hi,bs,ctx_hi", [
    (1, 1, 16, 5), (1, 300, 128, 1000), (7, 4, 64, 4096), (33, 1, 32, 200), (512, 5, 16, 900),
    (513, 40, 64, 300), (1500, 9, 128, 999), (8192, 2, 16, 64), (3, 9000, 16, 100)])
@pytest.mark.parametrize("release", [0.0, 0.3])
def test_plan(n, run_hi, bs, ctx_hi, release):
    check_plan(plan_case(n + run_hi, n, run_hi, bs, ctx_hi, release))


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("n,run_hi", [(5, 60), (70, 90), (600, 30)])
def test_plan_short_of_pages_serves_a_prefix(seed, n, run_hi):
    check_plan(plan_case(seed, n, run_hi, 16, 200, release=0.1 * (seed % 2), short=True))


def test_plan_total_wider_than_the_table_is_not_served():
    c = plan_case(5, 40, 100, 16, 300, width_cut=4)
    assert any(-(-(x + b - a) // 16) > len(c["tables"][0])
               for x, a, b in zip(c["cached"], c["cu"], c["cu"][1:]))
    check_plan(c)


def test_plan_everything_empty():
    c = dict(cached=[0, 0], cu=[0, 0, 0], tables=[[], []], held=[0, 0], free=[], count=0, bs=16, t=0,
             release=None)
    check_plan(c)


def test_plan_repeats_and_takes_released_pages_first():
    c = dict(cached=[20, 0, 33], cu=[0, 0, 40, 41], tables=[[4, 5, -1], [-1] * 3, [6, 7, 8]],
             held=[2, 0, 3], free=[0, 1, -9, -9, -9], count=2, bs=16, t=41, release=[1, 0, 0])
    first = run_plan(c)
    assert first[0] == [0, 40, 34] and first[1] == [0, 3, 3] and first[2] == [1]
    assert first[5][1] == [5, 4, 1]  # the last released page first
    assert run_plan(c) == first


def test_plan_rows_past_the_runs_have_no_slot():
    c = dict(cached=[3], cu=[0, 2], tables=[[9]], held=[1], free=[], count=0, bs=16, t=5, release=None)
    got = run_plan(c)
    assert got[4] == [9 * 16 + 3, 9 * 16 + 4, -1, -1, -1]


@pytest.mark.parametrize("spoil", ["held_wide", "held_negative", "cached_negative", "cached_unheld",
                                   "cu_past", "count_over"])
def test_plan_reports_lengths_that_cannot_be(spoil):
    c = plan_case(3, 6, 20, 16, 100)
    if spoil == "held_wide":
        c["held"][2] = 10000
    elif spoil == "held_negative":
        c["held"][2] = -1
    elif spoil == "cached_negative":
        c["cached"][2] = -5
    elif spoil == "cached_unheld":
        c["cached"][2] = c["held"][2] * 16 + 1
    elif spoil == "cu_past":
        c["cu"][6] += 50
    else:
        c["count"] = len(c["free"]) + 1
    run_plan(c)
    assert kda().read_device_status() == INVALID
    check_plan(plan_case(3, 6, 20, 16, 100))  # and the next call is sound


# ---------------------------------------------------------------------------------------- append
def pool(seed, pages, heads, bs, low=-3, high=3):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randn(pages, heads, bs, 128, generator=g) * 60
    scale = torch.exp2(torch.randint(low, high, (pages, heads), generator=g).float())
    return codes.clamp(-448, 448).to(E4M3), scale


def slots_of(seed, runs, ctx, bs, spare=2):
    """Slots of runs of tokens at positions ctx .. on shuffled pages."""
    r = random.Random(seed)
    need = [-(-(c + k) // bs) for c, k in zip(ctx, runs)]
    pages = list(range(sum(need) + spare))
    r.shuffle(pages)
    slots = []
    for c, k, m in zip(ctx, runs, need):
        mine = [pages.pop() for _ in range(m)]
        slots += [mine[p // bs] * bs + p % bs for p in range(c, c + k)]
    return slots, sum(need) + spare


def check_append(k, v, slots, kc, vc, ks, vs):
    dev = [x.to(DEV) for x in (kc, vc, ks, vs)]
    kda().paged_append(k.to(DEV) if k.device.type == "cpu" else k,
                       v.to(DEV) if v.device.type == "cpu" else v, i32(slots), *dev)
    for name, x, c0, s0, c1, s1 in (("k", k, kc, ks, dev[0], dev[2]), ("v", v, vc, vs, dev[1], dev[3])):
        codes, scale = c0.double().numpy().copy(), s0.double().numpy().copy()
        ref.append(x.cpu().double().numpy(), slots, codes, scale)
        np.testing.assert_array_equal(s1.cpu().double().numpy(), scale, err_msg=name)
        np.testing.assert_array_equal(c1.cpu().double().numpy(), codes, err_msg=name)
    assert kda().read_device_status() == 0


@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("heads,runs,ctx", [
    (1, [1], [0]), (2, [1], [37]), (3, [1, 0, 4, 8, 9, 2], [0, 5, 15, 60, 127, 128]),
    (2, [300, 1, 129], [0, 64, 3]), (8, [1] * 70, list(range(70)))])
def test_append(bs, heads, runs, ctx):
    slots, pages = slots_of(bs + heads, runs, ctx, bs)
    g = torch.Generator().manual_seed(heads)
    size = torch.exp(2 * torch.randn(sum(runs), heads, 1, generator=g))
    k, v = ((torch.randn(sum(runs), heads, 128, generator=g) * size).to(torch.bfloat16) for _ in "kv")
    check_append(k, v, slots, *pool(1, pages, heads, bs)[:1], *pool(2, pages, heads, bs)[:1],
                 pool(1, pages, heads, bs)[1], pool(2, pages, heads, bs)[1])


@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("heads,runs,ctx", [
    (3, [3000, 1, 700, 5000, 0, 13, 2100], [7, 90, 0, 300, 0, 125, 64]),
    (8, [9001, 4100], [13, 128]), (1, [3] * 3000, [k % 300 for k in range(3000)])])
def test_append_many_tokens(bs, heads, runs, ctx):
    """Blocks of 32 to 128 tokens: groups that end in the next block's tokens, many short ones."""
    slots, pages = slots_of(bs + heads, runs, ctx, bs)
    g = torch.Generator().manual_seed(heads)
    k, v = (torch.randn(sum(runs), heads, 128, generator=g).to(torch.bfloat16) for _ in "kv")
    check_append(k, v, slots, *pool(1, pages, heads, bs)[:1], *pool(2, pages, heads, bs)[:1],
                 pool(1, pages, heads, bs)[1], pool(2, pages, heads, bs)[1])


@pytest.mark.parametrize("m", [1, 8, 9, 40])
def test_append_growing_scale_codes_held_tokens_again(m):
    """The scale grows by up to 2^14: held codes fall into the subnormals and to zero."""
    slots = [3 * 64 + 20 + i for i in range(m)]
    for power in (0, 1, 5, 14):
        k = torch.full((m, 2, 128), 448.0 * 2.0 ** power).to(torch.bfloat16)
        v = -k
        kc, _ = pool(5, 5, 2, 64)
        vc, _ = pool(6, 5, 2, 64)
        one = torch.ones(5, 2)
        check_append(k, v, slots, kc, vc, one, one.clone())


def test_append_scale_that_is_no_power_of_two():
    slots = [70, 71, 72]
    g = torch.Generator().manual_seed(3)
    k = torch.randn(3, 1, 128, generator=g).to(torch.bfloat16)
    kc, _ = pool(5, 3, 1, 64)
    scale = torch.full((3, 1), 0.3)
    dev = [x.to(DEV) for x in (kc, kc, scale, scale)]
    kda().paged_append(k.to(DEV), k.to(DEV), i32(slots), *dev)
    # x / fp32(0.3) rounded to fp32 and then to e4m3, as the call does
    want = (k.float() / scale[0, 0]).to(E4M3).float()
    assert torch.equal(dev[0].float().cpu()[1, 0, 6:9], want[:, 0])
    assert torch.equal(dev[2].cpu(), scale)
    assert torch.equal(dev[0].float().cpu()[1, 0, :6], kc.float()[1, 0, :6])


def test_append_edges_of_the_scale():
    """Maxima at and beside 448 2^e, zeros, subnormal and huge inputs."""
    top = torch.tensor([448.0, 450.0, 446.0, 0.0, 1e-38, 9e-41, 3e38, 1.0]).to(torch.bfloat16)
    for value in top:
        k = torch.zeros(2, 1, 128, dtype=torch.bfloat16)
        k[0, 0, 7], k[1, 0, 99] = value, -value / 3
        kc, ks = pool(1, 2, 1, 16)
        check_append(k, -k, [16, 17], kc, kc, ks, ks.clone())


def test_append_nan_and_infinities_become_nan():
    k = torch.randn(12, 2, 128).to(torch.bfloat16)
    k[0, 0, 3], k[5, 1, 9], k[6, 1, 10] = float("nan"), float("inf"), -float("inf")
    kc, ks = pool(1, 3, 2, 16)
    check_append(k, k, list(range(32, 44)), kc, kc, ks, ks.clone())


def test_append_strided_views_and_skipped_tokens():
    """Runs without a slot (a request the plan did not serve) before, between and after others."""
    x = torch.randn(40, 13, 128, device=DEV).to(torch.bfloat16)
    slots = [-1] * 3 + list(range(64, 84)) + [-1] * 2 + list(range(9, 21)) + [-1] * 3
    kc, ks = pool(1, 4, 3, 64)
    check_append(x[:, 5:8], x[:, 10:13], slots, kc, kc, ks, ks.clone())


def test_append_slot_outside_the_pool_is_reported():
    x = torch.randn(3, 2, 128, device=DEV).to(torch.bfloat16)
    kc, ks = pool(1, 2, 2, 16)
    dev = [t.to(DEV) for t in (kc, kc, ks, ks)]
    kda().paged_append(x, x, i32([32, 33, 5]), *dev)
    assert kda().read_device_status() == INVALID
    assert torch.equal(dev[0].float().cpu()[1], kc.float()[1])


# ------------------------------------------------------------------------------------- attention
def attend_case(seed, runs, ctx, heads, kv, bs, q_size=1.5, low=-2, high=2, spoil=True, spare=1):
    g = torch.Generator().manual_seed(seed)
    need = [max(0, -(-c // bs)) for c in ctx]
    width = max(need + [1]) + spare
    perm = torch.randperm(sum(need) + 2, generator=g).tolist()
    tables = [[-1] * width for _ in ctx]
    for i, m in enumerate(need):
        for j in range(m):
            tables[i][j] = perm.pop()
    pages = sum(need) + 2
    kc, ks = ((torch.randn(pages, kv, bs, 128, generator=g) * 8).to(E4M3),
              torch.exp2(torch.randint(low, high, (pages, kv), generator=g).float()) / 8)
    vc, vs = ((torch.randn(pages, kv, bs, 128, generator=g) * 8).to(E4M3),
              torch.exp2(torch.randint(low, high, (pages, kv), generator=g).float()) / 8 * 1.17)
    if spoil:  # what a page holds beyond its context does not matter: NaN there
        raw_k, raw_v = kc.view(torch.uint8), vc.view(torch.uint8)
        for i, c in enumerate(ctx):
            if c > 0 and c % bs:
                raw_k[tables[i][c // bs], :, c % bs:] = 0x7F
                raw_v[tables[i][c // bs], :, c % bs:] = 0xFF
        for page in perm:
            raw_k[page], raw_v[page] = 0x7F, 0x7F
            ks[page], vs[page] = float("nan"), float("inf")
    q = (torch.randn(sum(runs), heads, 128, generator=g) * q_size).to(torch.bfloat16)
    return dict(q=q, cu=cu_of(runs), tables=tables, ctx=ctx, kc=kc, vc=vc, ks=ks, vs=vs,
                max_run=max(runs + [0]))


def attend(c, **kw):
    d = {k: c[k].to(DEV) for k in ("kc", "vc", "ks", "vs")}
    return kda().paged_attention(c["q"].to(DEV), i32(c["cu"]), i32(c["tables"]), i32(c["ctx"]), d["kc"],
                                 d["vc"], d["ks"], d["vs"], c["max_run"], **kw)


def check_attend(c, **kw):
    """The bound.  The output is rounded to bf16 (2^-9 |o|).  Weights are held to 8 bits or more
    (2^-9 relative each, so at most 2^-9 of the weighted mean of |v|, and 2^-9 |o| through their
    sum) down to 2^-16 of the row's largest; a smaller one is held within 2^-25 of the largest,
    which is at most their sum: 2^-25 of the sum of |v|.  Scores are fp32 sums of 128 exact products: within 2^-24 * 128 * sum |q||k| scale, a
    relative change of the weights as large, doubled for weights and sum."""
    out = attend(c, **kw)
    o, spread, top, most = ref.attention(c["q"], c["cu"], c["tables"], c["ctx"], c["kc"], c["vc"], c["ks"],
                                   c["vs"], **{k: v for k, v in kw.items() if k == "sm_scale"})
    got = out.double().cpu().numpy()
    bound = 2.0 ** -8 * np.abs(o) + (2.0 ** -9 + 2.0 ** -16 * top) * spread + 2.0 ** -25 * most + 1e-30
    worst = (np.abs(got - o) / bound).max(initial=0.0)
    assert np.isfinite(got).all() and worst <= 1, worst
    assert kda().read_device_status() == 0
    return out


@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("heads,kv", [(1, 1), (4, 4), (6, 2), (8, 1), (16, 2)])
def test_attention_decode(bs, heads, kv):
    ctx = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1000, 700]
    check_attend(attend_case(heads, [1] * len(ctx), ctx, heads, kv, bs))


@pytest.mark.parametrize("heads,kv,runs,ctx", [
    (8, 1, [1, 2, 3, 4, 8, 0, 5], [1, 2, 130, 128, 8, 77, 600]),
    (5, 1, [13, 1], [300, 1]),                   # 65 rows: a second row tile with one row
    (32, 1, [2, 4], [129, 260]),                 # 64 and 128 rows
    (40, 1, [3], [200]),                         # a tile ends inside a token's heads
    (64, 1, [1, 3], [300, 90]),
    (160, 1, [1], [300]),                        # more heads than a tile has rows
    (2, 2, [200, 33], [200, 517]),               # a prefill from nothing, a chunk over a prefix
    (12, 3, [65, 1, 64], [400, 1025, 64])])
@pytest.mark.parametrize("bs", [16, 64])
def test_attention_runs(heads, kv, runs, ctx, bs):
    check_attend(attend_case(sum(runs), runs, ctx, heads, kv, bs))


def test_attention_rows_that_see_nothing_are_zero():
    """A context shorter than the run (its first tokens see no key), an empty one, empty runs."""
    c = attend_case(3, [4, 2, 0, 5, 1], [2, 0, 40, 1, 0], 4, 2, 16)
    out = check_attend(c)
    assert (out[:2] == 0).all() and (out[4:6] == 0).all() and (out[6:10] == 0).all()
    assert (out[2:4] != 0).any() and (out[10] != 0).any() and (out[11] == 0).all()


@pytest.mark.parametrize("runs,heads,kv", [([1], 8, 1), ([4], 16, 1), ([1, 1, 1], 4, 2)])
def test_attention_long_contexts_are_split_and_joined(runs, heads, kv):
    ctx = [20011, 128 * 90, 6001][:len(runs)]
    check_attend(attend_case(11, runs, ctx, heads, kv, 64))


def test_attention_many_ragged_requests():
    r = random.Random(2)
    n = 200
    ctx = [r.choice([1, 50, 128, 129, 300, 1500]) for _ in range(n)]
    runs = [min(c, r.randint(0, 3)) for c in ctx]
    check_attend(attend_case(2, runs, ctx, 8, 2, 32))


# one layout of every tile the kernels have: 8, 16, 32, 64, 128 and 256 rows
ROWS = [(4, 1, 2), (8, 1, 2), (16, 1, 2), (16, 1, 4), (16, 1, 7), (8, 1, 40)]  # heads, kv, run


@pytest.mark.parametrize("heads,kv,run", ROWS)
@pytest.mark.parametrize("bs", [16, 128])
def test_attention_short_contexts_back_to_back(heads, kv, run, bs):
    """Many units of one to three tiles, so that a block goes from one to the next all the time."""
    r = random.Random(run)
    runs = [r.randint(0, run) for _ in range(700)]
    runs[0] = run
    ctx = [k + r.choice([0, 1, 20, 100, 128, 250]) for k in runs]
    check_attend(attend_case(run, runs, ctx, heads, kv, bs))


@pytest.mark.parametrize("heads,kv,run", ROWS)
def test_attention_splits_of_every_tile(heads, kv, run):
    """Long units cut between blocks and joined, ragged ones among them, contexts shorter than runs."""
    check_attend(attend_case(run, [run, 1, 0, run, run], [9001, 700, 50, run - 1, 4 * 128 + 1], heads, kv, 64))


@pytest.mark.parametrize("heads,kv,run", ROWS)
@pytest.mark.parametrize("kw", [dict(q_size=30.0), dict(q_size=1e-3),
                                dict(q_size=0.05, low=-12, high=12)])
def test_attention_sizes_of_scores_and_scales(heads, kv, run, kw):
    check_attend(attend_case(run + 1, [run, 1], [1100, 401], heads, kv, 32, **kw))


def check_nan(c):
    """NaN exactly where the reference has it, everything else within the bound."""
    out = attend(c).double().cpu().numpy()
    o, spread, top, most = ref.attention(c["q"], c["cu"], c["tables"], c["ctx"], c["kc"], c["vc"],
                                         c["ks"], c["vs"])
    np.testing.assert_array_equal(np.isnan(out), np.isnan(o))
    fine = ~np.isnan(o)
    bound = 2.0 ** -8 * np.abs(o) + (2.0 ** -9 + 2.0 ** -16 * top) * spread + 2.0 ** -25 * most + 1e-30
    assert (np.abs(out - o)[fine] <= bound[fine]).all()
    assert kda().read_device_status() == 0


def put_nan(c, which, request, pos, channel):
    bs = c["kc"].shape[2]
    c[which].view(torch.uint8)[c["tables"][request][pos // bs], :, pos % bs, channel] = 0x7F


@pytest.mark.parametrize("heads,kv,run", ROWS)
def test_attention_nan_of_a_masked_key_stays_out(heads, kv, run):
    """NaN in a run token's key or value reaches that token and later ones, not the earlier ones
    that share its tile; in a value, its channel only."""
    ctx = [700, 300 + run]
    for which, channel in (("vc", 5), ("vc", 127), ("kc", 9)):
        c = attend_case(run, [run, run], ctx, heads, kv, 32, spoil=False)
        put_nan(c, which, 0, ctx[0] - 1, channel)             # the last token of a run
        put_nan(c, which, 1, ctx[1] - 1 - run // 2, channel)  # one in the middle
        check_nan(c)
    c = attend_case(run, [run, run], ctx, heads, kv, 32, spoil=False)
    put_nan(c, "vc", 0, 40, 77)  # seen by every row of a request
    check_nan(c)


@pytest.mark.parametrize("heads,kv,run", ROWS)
def test_attention_nan_and_infinite_queries_stay_in_their_row(heads, kv, run):
    c = attend_case(run, [run], [333], heads, kv, 64)
    c["q"][run - 1, heads - 1, 3] = float("nan")
    c["q"][0, 1, 100] = float("inf")
    out = attend(c)
    bad = torch.zeros(run, heads, dtype=torch.bool)
    bad[run - 1, heads - 1] = bad[0, 1] = True
    assert torch.equal(out.isnan().all(-1).cpu(), bad) and torch.equal(out.isnan().any(-1).cpu(), bad)
    c["q"][bad] = 0
    assert torch.equal(out[~bad], check_attend(c)[~bad])


def test_attention_decodes_next_to_a_prompt():
    """One call with a chunk of a prompt and single tokens."""
    check_attend(attend_case(21, [150, 1, 1, 40, 1], [400, 900, 3, 40, 2000], 8, 2, 64))


def test_cache_beyond_four_gigabytes():
    """Pages whose byte offsets pass 32 bits."""
    pages = (1 << 32) // (2 * 16 * 128) + 40
    kc = torch.zeros(pages, 2, 16, 128, dtype=torch.uint8, device=DEV).view(E4M3)
    vc = torch.zeros(pages, 2, 16, 128, dtype=torch.uint8, device=DEV).view(E4M3)
    ks, vs = torch.zeros(pages, 2, device=DEV), torch.zeros(pages, 2, device=DEV)
    table = [pages - 1, 3, pages - 20]
    slots = [table[i // 16] * 16 + i % 16 for i in range(40)]
    g = torch.Generator().manual_seed(4)
    k, v = (torch.randn(40, 2, 128, generator=g).to(torch.bfloat16) for _ in "kv")
    kda().paged_append(k.to(DEV), v.to(DEV), i32(slots), kc, vc, ks, vs)
    q = torch.randn(1, 4, 128, generator=g).to(torch.bfloat16)
    out = kda().paged_attention(q.to(DEV), i32([0, 1]), i32([table]), i32([40]), kc, vc, ks, vs, 1)
    few = dict(q=q, cu=[0, 1], tables=[[0, 1, 2]], ctx=[40], max_run=1,
               **{n: t.view(torch.uint8)[table].cpu().view(E4M3) for n, t in (("kc", kc), ("vc", vc))},
               **{n: t[table].cpu() for n, t in (("ks", ks), ("vs", vs))})
    assert (few["ks"] > 0).all() and few["kc"].float().abs().amax() > 200
    assert torch.equal(out, check_attend(few))


@pytest.mark.parametrize("q_size", [1e-3, 30.0])
def test_attention_flat_and_peaked(q_size):
    check_attend(attend_case(7, [2, 1], [900, 401], 8, 2, 64, q_size=q_size))


def test_attention_scales_that_differ_widely():
    """Page scales spread over 2^24, as pages of very different size."""
    check_attend(attend_case(8, [3, 1], [700, 300], 4, 2, 16, q_size=0.05, low=-12, high=12))


def test_attention_a_heavy_first_key_and_a_long_light_tail():
    """Half of the weight on one key, the other half over 16K keys of 2^-14 of it each: small
    weights keep their relative precision."""
    c = attend_case(9, [1], [16385], 4, 1, 64, spoil=False)
    c["q"][:] = 0
    c["q"][:, :, 0] = 1.0
    kc = torch.zeros(c["kc"].shape)
    page = c["tables"][0][0]
    kc[page, :, 0, 0] = 112.0
    c["kc"], c["ks"] = kc.to(E4M3), torch.ones_like(c["ks"])
    want = 14 * np.log(2.0) / 112.0
    vc = torch.ones(c["vc"].shape)
    vc[page, :, 0] = -1.0
    c["vc"], c["vs"] = vc.to(E4M3), torch.ones_like(c["vs"])
    out = attend(c, sm_scale=float(np.float32(want)))
    o, spread, _, _ = ref.attention(c["q"], c["cu"], c["tables"], c["ctx"], c["kc"], c["vc"], c["ks"],
                                 c["vs"], sm_scale=float(np.float32(want)))
    # weights 2^-14 of the largest within 2^-9: |o| is about 0, so the bound is the spread's
    assert np.abs(out.double().cpu().numpy() - o).max() <= 2.0 ** -8 * spread.max()


def test_attention_equal_rows_of_a_group_and_repeats_are_bit_exact():
    c = attend_case(12, [2, 1, 3], [5000, 130, 3000], 8, 2, 32)
    c["q"][:] = c["q"][:, :1]
    a, b = attend(c), attend(c)
    assert torch.equal(a, b)


def test_attention_strided_queries_scale_and_buffers():
    c = attend_case(13, [2, 3], [100, 260], 4, 2, 16)
    x = torch.randn(5, 9, 128, device=DEV).to(torch.bfloat16)
    x[:, 2:6] = c["q"].to(DEV)
    d = {k: c[k].to(DEV) for k in ("kc", "vc", "ks", "vs")}
    need = kda().paged_attention_workspace_bytes(4, 2, 3)
    ws = torch.full((max(need, 1),), 255, dtype=torch.uint8, device=DEV)  # contents are ignored
    out = torch.empty(5, 4, 128, dtype=torch.bfloat16, device=DEV)
    got = kda().paged_attention(x[:, 2:6], i32(c["cu"]), i32(c["tables"]), i32(c["ctx"]), d["kc"],
                                d["vc"], d["ks"], d["vs"], 3, sm_scale=0.2, out=out, workspace=ws)
    assert got is out
    assert torch.equal(out, check_attend(c, sm_scale=0.2))


@pytest.mark.parametrize("spoil", ["page_high", "page_negative", "wide", "run"])
def test_attention_reports_what_points_outside(spoil):
    c = attend_case(14, [2, 1], [100, 70], 4, 2, 16)
    if spoil == "page_high":
        c["tables"][0][3] = 10 ** 6
    elif spoil == "page_negative":
        c["tables"][1][0] = -3
    elif spoil == "wide":
        c["ctx"][0] = 16 * len(c["tables"][0]) + 1
    else:
        c["max_run"] = 1
    attend(c)
    assert kda().read_device_status() == INVALID
    check_attend(attend_case(14, [2, 1], [100, 70], 4, 2, 16))


def test_attention_on_another_stream_and_in_a_graph():
    c = attend_case(15, [2, 1, 4], [3000, 70, 515], 8, 2, 64)
    want = check_attend(c)
    d = {k: c[k].to(DEV) for k in ("kc", "vc", "ks", "vs")}
    q, cu, tables, ctx = c["q"].to(DEV), i32(c["cu"]), i32(c["tables"]), i32(c["ctx"])
    out = torch.empty_like(q)
    ws = torch.empty(max(1, kda().paged_attention_workspace_bytes(8, 2, 4)), dtype=torch.uint8, device=DEV)
    call = lambda **kw: kda().paged_attention(q, cu, tables, ctx, d["kc"], d["vc"], d["ks"], d["vs"], 4,  # noqa: E731
                                              out=out, workspace=ws, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call(stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    # lengths change on the device, the graph stays
    ctx.copy_(i32([900, 65, 300]))
    graph.replay()
    torch.cuda.synchronize()
    c["ctx"] = [900, 65, 300]
    assert torch.equal(out, check_attend(c))


# ------------------------------------------------------------------------------------------ verify
def verify_case(seed, runs, vocab, dtype, drafted=True, close=0.6):
    g = torch.Generator().manual_seed(seed)
    t = sum(runs)
    z = torch.randn(t, vocab, generator=g) * 2
    p = torch.softmax(z, -1).to(dtype)
    q = torch.softmax(z + close * torch.randn(t, vocab, generator=g), -1).to(dtype) if drafted else None
    tokens = torch.zeros(t, dtype=torch.int32)
    tokens[1:] = torch.multinomial((q if drafted else p).float(), 1, generator=g)[:-1, 0].to(torch.int32)
    return dict(p=p, q=q, tokens=tokens, cu=cu_of(runs), u=torch.rand(t, generator=g),
                e=torch.empty(len(runs), vocab).exponential_(generator=g))


def check_verify(c):
    f = lambda x: None if x is None else x.float().numpy()  # noqa: E731
    want = ref.verify(f(c["p"]), f(c["q"]), c["tokens"].tolist(), c["cu"], f(c["u"]), f(c["e"]))
    got = kda().verify_draft(c["p"].to(DEV), c["tokens"].to(DEV), i32(c["cu"]), c["u"].to(DEV),
                             c["e"].to(DEV), draft_probs=None if c["q"] is None else c["q"].to(DEV))
    for name, g, w in zip(("commit", "next", "out"), got, want):
        assert g.tolist() == w, name
    return want


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("drafted", [True, False])
@pytest.mark.parametrize("vocab", [1, 3, 64, 1001, 4096, 50002, 32000])
def test_verify(dtype, drafted, vocab):
    c = verify_case(vocab, [4, 1, 0, 8, 2, 5, 1], vocab, dtype, drafted)
    check_verify(c)
    assert kda().read_device_status() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("drafted", [True, False])
@pytest.mark.parametrize("n,vocab", [(28, 2000), (29, 2001), (131, 512), (131, 999)])
def test_verify_many_requests(dtype, drafted, n, vocab):
    check_verify(verify_case(n, [k % 4 for k in range(n)], vocab, dtype, drafted))
    assert kda().read_device_status() == 0


def test_verify_every_draft_holds_and_none():
    c = verify_case(1, [40, 33, 70], 500, torch.float32, close=0.0)
    c["u"][:] = 0.5
    assert check_verify(c)[0] == [40, 33, 70]
    c["u"][:] = 0.999999
    c["p"], c["q"] = c["p"] * 0.5, c["q"]
    assert check_verify(c)[0] == [1, 1, 1]
    c["u"][:] = 0.0
    c["u"][60] = 0.9  # the second run's draft 20
    assert check_verify(c)[0][1] == 21


def test_verify_ties_go_to_the_lowest_token():
    v = 5000
    c = verify_case(2, [1, 2, 1], v, torch.float32)
    c["p"][:] = 1.0 / v
    c["q"][:] = 1.0 / v
    c["e"][:] = 1.0
    c["e"][0, [4000, 17, 4999]] = 0.25
    c["u"][:] = 0.0
    assert check_verify(c)[1] == [17, 0, 0]


def test_verify_nothing_left_of_the_difference_falls_back_to_the_target():
    c = verify_case(3, [3, 2], 1000, torch.float32)
    c["q"] = c["p"].clone()
    c["q"][:, :] = c["p"] * 1.5
    c["u"][:] = 0.9
    assert check_verify(c)[0] == [1, 1]


def test_verify_zero_and_infinite_noise_and_zero_rows():
    c = verify_case(4, [1, 1, 1], 777, torch.float32)
    c["e"][0, 300] = 0.0
    c["e"][1, :] = float("inf")
    c["p"][2] = 0.0
    want = check_verify(c)
    assert want[1][0] == 300 and want[1][2] == 0


def test_verify_draft_outside_the_vocabulary_falls_and_is_reported():
    c = verify_case(5, [3, 3], 100, torch.float32)
    c["u"][:] = 0.0
    c["tokens"][2], c["tokens"][4] = 100, -1
    want = check_verify(c)
    assert want[0] == [2, 1]
    assert kda().read_device_status() == INVALID


def test_verify_probabilities_follow_the_target():
    """With random u and e, first accepted token or replacement is distributed as the target: over
    40,000 requests of one draft each, every frequency is within 5 standard deviations."""
    n, v = 40000, 8
    g = torch.Generator(device=DEV).manual_seed(1)
    p = torch.tensor([.3, .05, .2, .1, .02, .13, .15, .05], device=DEV)
    q = torch.tensor([.1, .25, .1, .1, .2, .05, .15, .05], device=DEV)
    tokens = torch.zeros(2 * n, dtype=torch.int32, device=DEV)
    tokens[1::2] = torch.multinomial(q, n, replacement=True, generator=g).to(torch.int32)
    cu = (2 * torch.arange(n + 1, device=DEV)).to(torch.int32)
    _, _, out = kda().verify_draft(p.repeat(2 * n, 1), tokens, cu, torch.rand(2 * n, device=DEV, generator=g),
                                   torch.empty(n, v, device=DEV).exponential_(generator=g),
                                   draft_probs=q.repeat(2 * n, 1))
    freq = torch.bincount(out[::2].long(), minlength=v).double().cpu() / n
    want = p.double().cpu()
    assert ((freq - want).abs() <= 5 * (want * (1 - want) / n).sqrt()).all(), freq


# ----------------------------------------------------------------------------------------- together
def test_speculative_step_example(capsys):
    """Plan, append, attention, decode window and verification as a serving loop runs them; the KDA
    states end up where the kept tokens alone lead."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "speculative_step.py")
    spec = importlib.util.spec_from_file_location("speculative_step", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    example.main(9)
    assert "states match" in capsys.readouterr().out
