"""Cases of the paged serving operators: page plan, cache append, attention over the 8-bit cache,
verification of drafted tokens.

One speculative decoding step of a hybrid model (KDA layers next to full-attention layers that
keep keys and values in pages) runs, in this order,

  plan     block tables, token positions and cache slots from the requests' lengths
  append   the step's keys and values into the pages, 8 bits with a scale per (page, head)
  attend   every run token's attention over the request's pages
  verify   accepted drafts and the next token, from the target's probabilities and given
           random numbers; its counts are what ``decode_window(commit=...)`` takes

Pages hold ``bs`` tokens of one head contiguously: caches [pages, Hkv, bs, 128] in e4m3, scales
fp32 [pages, Hkv].  A page's scale is a power of two: the smallest s >= 2^-100 with
amax <= 448 s.
"""
import math

import torch

own = False

D = 128
DEV = "cuda"
E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # the smallest call: one request, one token, a short prompt; latency is what counts
        dict(name="attend_one", op="attend", n=1, run_lo=1, run_hi=1, heads=16, kv_heads=2, bs=64,
             ctx_lo=257, ctx_hi=257),
        # an ordinary decode batch without drafts, contexts spread over 512 .. 16K tokens
        dict(name="attend_decode_64", op="attend", n=64, run_lo=1, run_hi=1, heads=32, kv_heads=8,
             bs=64, ctx_lo=512, ctx_hi=16384),
        # a speculative batch: ragged runs of 1 to 8 tokens, 8 query heads to a key head
        dict(name="attend_window_128", op="attend", n=128, run_lo=1, run_hi=8, heads=32,
             kv_heads=4, bs=32, ctx_lo=2048, ctx_hi=8192),
        # one long request (256K tokens, 16 heads on one key head): few rows, a long axis
        dict(name="attend_long_256k", op="attend", n=1, run_lo=4, run_hi=4, heads=16, kv_heads=1,
             bs=128, ctx_lo=262144, ctx_hi=262144),
        # chunked prefill: about a thousand new tokens each on top of a cached prefix
        dict(name="attend_chunk", op="attend", n=3, run_lo=900, run_hi=1100, heads=32, kv_heads=8,
             bs=64, ctx_lo=6000, ctx_hi=8192),
        # a decode step's keys and values, 1 to 4 tokens a request, into pages already begun
        dict(name="append_step_256", op="append", n=256, run_lo=1, run_hi=4, kv_heads=8, heads=32,
             bs=64, ctx_lo=1, ctx_hi=4096),
        # the keys and values of a prefill of 4 x 8192 tokens
        dict(name="append_prefill_32k", op="append", n=4, run_lo=8192, run_hi=8192, kv_heads=8,
             heads=32, bs=64, ctx_lo=0, ctx_hi=0),
        # a decode step of 64 requests with 4 tokens each; a few finish and give their pages back
        dict(name="plan_step_64", op="plan", n=64, run_lo=4, run_hi=4, bs=64, ctx_lo=1,
             ctx_hi=16384, release=0.05),
        # a large mixed batch: 512 requests, ragged prefill chunks up to 512 tokens
        dict(name="plan_mixed_512", op="plan", n=512, run_lo=1, run_hi=512, bs=16, ctx_lo=1,
             ctx_hi=8192, release=0.1),
        # one request with three drafts and a small vocabulary
        dict(name="verify_one", op="verify", n=1, run_lo=4, run_hi=4, vocab=32000, drafted=True,
             dtype="float32"),
        # a serving batch: 64 requests, up to 7 drafts each, a large vocabulary
        dict(name="verify_64", op="verify", n=64, run_lo=1, run_hi=8, vocab=131072, drafted=True,
             dtype="float32"),
        # drafts without probabilities (prompt lookup: certain ones), an odd vocabulary, bf16
        dict(name="verify_lookup_odd", op="verify", n=19, run_lo=2, run_hi=6, vocab=50001,
             drafted=False, dtype="bfloat16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "plan", "verify"])
    bs = rng.choice([16, 32, 64, 128])
    if op == "attend":
        kv, group = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 4, 5, 8, 16])
        if rng.random() < 0.25:  # prefill chunks over a prefix
            group = min(group, 32 // kv)
            n, lo = rng.randint(1, 3), _log(rng, 65, 900)
            hi, ctx = lo + rng.randint(0, 150), _log(rng, 1200, 7000)
        else:
            n, lo = _log(rng, 1, 128), rng.randint(1, 4)
            hi = lo + rng.randint(0, 4)
            ctx = _log(rng, 16, max(64, min(262144, 262144 // n)))
        return dict(op=op, n=n, run_lo=lo, run_hi=hi, heads=kv * group, kv_heads=kv, bs=bs,
                    ctx_lo=max(hi, ctx // rng.choice([1, 2, 8])), ctx_hi=max(hi, ctx))
    if op == "append":
        n = _log(rng, 1, 256)
        lo = _log(rng, 1, max(1, 16384 // n))
        return dict(op=op, n=n, run_lo=lo, run_hi=lo + rng.randint(0, lo), bs=bs,
                    kv_heads=rng.choice([1, 2, 3, 4, 8]), heads=8, ctx_lo=0,
                    ctx_hi=rng.randint(1, 2048))
    if op == "plan":
        n = _log(rng, 1, 512)
        return dict(op=op, n=n, run_lo=rng.randint(0, 1), run_hi=_log(rng, 1, 512), bs=bs, ctx_lo=1,
                    ctx_hi=_log(rng, 16, 8192), release=rng.choice([0.0, 0.05, 0.3]))
    return dict(op=op, n=_log(rng, 1, 64), run_lo=rng.randint(0, 2), run_hi=rng.randint(2, 8),
                vocab=_log(rng, 1000, 131072), drafted=rng.random() < 0.6,
                dtype=rng.choice(["float32", "float32", "bfloat16"]))


def _released(case):
    """Which requests of a plan are done; their runs are empty."""
    gen = torch.Generator().manual_seed(case["n"])
    gone = torch.rand(case["n"], generator=gen) < case.get("release", 0.0)
    gone[0] = False
    return gone


def _lengths(case):
    """Host lists of run and context lengths (context: with the run), the same for every seed, so
    that ``work`` can count them."""
    gen = torch.Generator().manual_seed(case["n"] * 7919 + case["run_hi"])
    n, lo, hi = case["n"], case["run_lo"], case["run_hi"]
    runs = torch.randint(lo, hi + 1, (n,), generator=gen)
    runs[0] = hi
    runs[_released(case)] = 0
    if "ctx_hi" not in case:
        return runs.tolist(), None
    a, b = math.log(max(1, case["ctx_lo"])), math.log(max(1, case["ctx_hi"]))
    ctx = torch.exp(a + (b - a) * torch.rand(n, generator=gen, dtype=torch.float64)).round().long()
    if case["ctx_hi"] == 0:
        ctx.zero_()
    if case["op"] == "attend":  # the context holds the run
        ctx = torch.maximum(ctx, runs)
    return runs.tolist(), ctx.tolist()


def work(case):
    runs, ctx = _lengths(case)
    t, n = sum(runs), case["n"]
    if case["op"] == "attend":
        h, kv = case["heads"], case["kv_heads"]
        pages = sum(-(-c // case["bs"]) for c in ctx)
        seen = sum(r * c - r * (r - 1) // 2 for r, c in zip(runs, ctx))  # (token, key) pairs
        return {"bytes": sum(ctx) * kv * 2 * D + pages * (kv * 8 + 4) + t * h * D * 4 + n * 8,
                "flops": 4 * D * h * seen}
    if case["op"] == "append":
        kv = case["kv_heads"]
        pages = sum(-(-(c + r) // case["bs"]) - c // case["bs"] for r, c in zip(runs, ctx))
        # bf16 in, 8 bits out; a scale read and written for each page touched; the slots
        return {"bytes": t * kv * 2 * D * 3 + pages * kv * 16 + t * 4, "flops": t * kv * 2 * D * 2}
    if case["op"] == "plan":
        # lengths, counts and flags in and out; a table entry for each page of a token; the slots
        return {"bytes": n * 28 + t * 8 + sum(-(-(c + r) // case["bs"]) - c // case["bs"]
                                              for r, c in zip(runs, ctx)) * 8, "flops": 0}
    e = 4 if case["dtype"] == "float32" else 2
    rows = sum(1 for r in runs if r > 0)
    # a live request reads one row of the target, one of the random numbers and, where a draft
    # fell (about three requests in four here), one of the draft's
    return {"bytes": rows * case["vocab"] * (e + 4 + (0.75 * e if case["drafted"] else 0)) + t * 16,
            "flops": rows * case["vocab"] * 2}


# ------------------------------------------------------------------------------------ the inputs
def _cu(runs):
    return torch.tensor([0] + runs).cumsum(0).to(torch.int32).to(DEV)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _scale_of(amax):
    """Smallest power of two s >= 2^-100 with amax <= 448 s."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(min=-100)
    return torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, e, -100))


def _pages(gen, count, kv, bs, rows=None, at=None):
    """A pool of `count` pages: codes and scales of normal values whose size differs by head and
    page.  `rows` [m, kv, D] are put at the pages' first tokens `at` [m] before they are coded."""
    codes = torch.empty(count, kv, bs, D, dtype=E4M3, device=DEV)
    scale = torch.empty(count, kv, dtype=torch.float32, device=DEV)
    size = torch.exp(0.5 * torch.randn(1, kv, 1, 1, generator=gen, device=DEV))
    step = max(1, (1 << 27) // (kv * bs * D))
    for i in range(0, count, step):
        m = min(step, count - i)
        x = torch.randn(m, kv, bs, D, generator=gen, device=DEV) * size
        if rows is not None:
            here = (at >= i) & (at < i + m)
            x[at[here] - i, :, 0] = rows[here] * size[:, :, 0]
        s = _scale_of(x.abs().amax(dim=(2, 3)))
        codes[i:i + m] = (x / s[:, :, None, None]).to(E4M3)
        scale[i:i + m] = s
    return codes, scale


def _tables(gen, need, width, spare=0):
    """Tables of shuffled page numbers, -1 where a request has none, and the pages left over."""
    need = torch.as_tensor(need, device=DEV)
    total = int(need.sum()) + spare
    perm = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
    tables = torch.full((len(need), width), -1, dtype=torch.int32, device=DEV)
    tables[torch.arange(width, device=DEV)[None] < need[:, None]] = perm[:total - spare]
    return tables, perm[total - spare:].clone(), total


def _projection(gen, t, heads, kv):
    """A layer's fused projection and its views of queries, keys and values."""
    x = torch.randn(t, (heads + 2 * kv) * D, generator=gen, device=DEV).to(torch.bfloat16)
    x = x.view(t, heads + 2 * kv, D)
    return x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:]


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    runs, ctx = _lengths(case)
    t, n, op = sum(runs), case["n"], case["op"]
    s = dict(op=op, cu=_cu(runs), t=t, max_run=max(runs))
    if op == "verify":
        v, dt = case["vocab"], getattr(torch, case["dtype"])
        # peaked rows, the draft a blurred version of the target; three drafts in four hold
        z = torch.randn(t, v, generator=gen, device=DEV) * 2.5
        p = torch.softmax(z, -1)
        q = torch.softmax(z + 0.6 * torch.randn(t, v, generator=gen, device=DEV), -1)
        pick = torch.multinomial(q if case["drafted"] else p, 1, generator=gen)[:, 0]
        # run token i + 1 was drafted by row i; a run's first token is what came before
        tokens = torch.roll(pick, 1).to(torch.int32)
        if not case["drafted"]:  # a certain draft that the target likes about as often
            like = torch.rand(t, generator=gen, device=DEV) < 0.75
            at = torch.roll(tokens, -1).long()[:, None]
            p = torch.where(like[:, None], p * 0.1, p)
            p.scatter_add_(1, at, torch.where(like, 0.9, 0.0)[:, None])
        s |= dict(p=p.to(dt), q=q.to(dt) if case["drafted"] else None, tokens=tokens,
                  u=torch.rand(t, generator=gen, device=DEV),
                  e=torch.empty(n, v, device=DEV).exponential_(generator=gen))
        return s
    bs = case["bs"]
    if op == "attend":
        h, kv = case["heads"], case["kv_heads"]
        tables, _, count = _tables(gen, [-(-c // bs) for c in ctx], max(-(-c // bs) for c in ctx))
        # the first token of each request draws much of the attention, as it does in earnest
        lean = torch.nn.functional.normalize(torch.randn(kv, D, generator=gen, device=DEV), dim=-1)
        kc, ks = _pages(gen, count, kv, bs, rows=12 * lean[None].expand(n, -1, -1),
                        at=tables[:, 0].long())
        vc, vs = _pages(gen, count, kv, bs)
        q, _, _ = _projection(gen, t, h, kv)
        q.mul_(1.5).add_((6 * lean).repeat_interleave(h // kv, 0).to(torch.bfloat16))
        return s | dict(q=q, tables=tables, ctx=_i32(ctx), kc=kc, ks=ks, vc=vc, vs=vs)
    if op == "append":
        h, kv = case["heads"], case["kv_heads"]
        need = [-(-(c + r) // bs) for r, c in zip(runs, ctx)]
        tables, _, count = _tables(gen, need, max(need))
        kc, ks = _pages(gen, count, kv, bs)
        vc, vs = _pages(gen, count, kv, bs)
        _, k, v = _projection(gen, t, h, kv)
        row = torch.repeat_interleave(torch.arange(n, device=DEV), _i32(runs))
        pos = torch.arange(t, device=DEV) - s["cu"][row] + _i32(ctx)[row]
        slots = tables[row, pos // bs] * bs + (pos % bs).to(torch.int32)
        return s | dict(k=k, v=v, slots=slots, kc=kc, ks=ks, vc=vc, vs=vs)
    width = max(-(-(c + r) // bs) for r, c in zip(runs, ctx)) + 2
    held = [-(-c // bs) for c in ctx]
    tables, free, count = _tables(gen, held, width, spare=sum(runs) // bs + n)
    pool = torch.zeros(count, dtype=torch.int32, device=DEV)
    pool[:len(free)] = free
    release = _released(case).to(torch.int32).to(DEV)
    return s | dict(cached=_i32(ctx), held=_i32(held), tables=tables, pool=pool,
                    count=_i32([len(free)]), release=release, bs=bs)


# ------------------------------------------------------------------------------- one pass of each
def run(s):
    if own:
        import kimi_delta_attention_03_gb300 as kda
        if s["op"] == "attend":
            return kda.paged_attention(s["q"], s["cu"], s["tables"], s["ctx"], s["kc"], s["vc"],
                                       s["ks"], s["vs"], s["max_run"])
        if s["op"] == "append":
            kda.paged_append(s["k"], s["v"], s["slots"], s["kc"], s["vc"], s["ks"], s["vs"])
            return s["kc"], s["vc"], s["ks"], s["vs"]
        if s["op"] == "plan":
            got = kda.paged_plan(s["cached"], s["cu"], s["tables"], s["held"], s["pool"],
                                 s["count"], s["bs"], s["t"], release=s["release"])
            return (*got, s["tables"], s["pool"])
        return kda.verify_draft(s["p"], s["tokens"], s["cu"], s["u"], s["e"], draft_probs=s["q"])
    return {"attend": _attend, "append": _append, "plan": _plan, "verify": _verify}[s["op"]](s)


def _attend(s):
    q, cu, ctx, tables = s["q"], s["cu"].long(), s["ctx"].long(), s["tables"].long()
    kv, bs = s["kc"].shape[1], s["kc"].shape[2]
    t, h, _ = q.shape
    n, width = tables.shape
    g, m, keys = h // kv, s["max_run"], width * bs
    at = tables.clamp(min=0)
    k = s["kc"].view(torch.uint8)[at].view(E4M3).float()  # [n, width, kv, bs, D]
    v = s["vc"].view(torch.uint8)[at].view(E4M3).float()
    k, v = k * s["ks"][at][..., None, None], v * s["vs"][at][..., None, None]
    k = k.permute(0, 2, 4, 1, 3).reshape(n, kv, D, keys)
    v = v.permute(0, 2, 1, 3, 4).reshape(n, kv, keys, D)
    runs = cu[1:] - cu[:-1]
    i = torch.arange(m, device=q.device)
    src = (cu[:-1, None] + i[None]).clamp(max=t - 1)
    x = q[src].float().view(n, m, kv, g, D).permute(0, 2, 1, 3, 4).reshape(n, kv, m * g, D)
    z = (x @ k) * D ** -0.5
    last = (ctx - runs)[:, None] + i[None]  # run token i sees keys 0 .. last
    live = torch.arange(keys, device=q.device)[None, None] <= last[..., None]
    live = live & (torch.arange(keys, device=q.device) < ctx[:, None])[:, None]
    live = live[:, None, :, None].expand(n, kv, m, g, keys).reshape(n, kv, m * g, keys)
    z = torch.where(live, z, torch.full((), -math.inf, device=q.device))
    top = z.amax(-1, keepdim=True)
    w = torch.exp(z - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    total = w.sum(-1, keepdim=True)
    o = (w @ v) / torch.where(total > 0, total, torch.ones_like(total))
    o = o.view(n, kv, m, g, D).permute(0, 2, 1, 3, 4).reshape(n, m, h, D)
    row = torch.searchsorted(cu[1:], torch.arange(t, device=q.device), right=True)
    return o[row, torch.arange(t, device=q.device) - cu[row]].to(torch.bfloat16)


def _append(s):
    slots, bs, n = s["slots"].long(), s["kc"].shape[2], s["cu"].numel() - 1
    page, off = slots // bs, slots % bs  # every slot is in use here
    begins = torch.cat([page.new_ones(1, dtype=torch.bool), page[1:] != page[:-1]])
    group = torch.cumsum(begins, 0) - 1  # tokens of one page, one after another
    most = slots.numel() // bs + 2 * n  # at most so many groups; what is over repeats the first
    at = torch.where(begins, group, most)
    pages = page.new_full((most + 1,), -1).scatter_(0, at, page)[:most]
    first = page.new_zeros(most + 1).scatter_(0, at, off)[:most]
    of = torch.where(pages >= 0, torch.arange(most, device=page.device), 0)
    spot = (page, off, group, pages[of], first[of], of)
    _append_one(s["k"].float(), s["kc"].view(torch.uint8), s["ks"], *spot)
    _append_one(s["v"].float(), s["vc"].view(torch.uint8), s["vs"], *spot)
    return s["kc"], s["vc"], s["ks"], s["vs"]


def _append_one(x, codes, scale, page, off, group, pages, first, of):
    amax = torch.where(x.isfinite(), x.abs(), torch.zeros_like(x)).amax(-1)
    amax = amax.new_zeros(len(pages), amax.shape[1]).index_reduce_(0, group, amax, "amax")[of]
    new, old = _scale_of(amax), scale[pages]
    begun = (first > 0)[:, None]
    new = torch.where(begun, torch.maximum(new, old), new)
    # the tokens that a page held before are coded again where its scale grew
    held = torch.arange(codes.shape[2], device=x.device) < first[:, None]
    grew = ((begun & (new > old))[:, :, None] & held[:, None])[..., None]
    was = codes[pages]
    again = (was.view(E4M3).float() * (old / new)[:, :, None, None]).to(E4M3).view(torch.uint8)
    codes[pages] = torch.where(grew, again, was)
    scale[pages] = new
    codes[page, :, off] = (x / scale[page][..., None]).to(E4M3).view(torch.uint8)


def _plan(s):
    bs, cu, tables, pool, t = s["bs"], s["cu"].long(), s["tables"], s["pool"], s["t"]
    n, width = tables.shape
    gone = s["release"] != 0
    runs = cu[1:] - cu[:-1]
    cached = torch.where(gone, 0, s["cached"].long())
    col = torch.arange(width, device=cu.device)
    back = gone[:, None] & (col < s["held"][:, None])  # pages given back, in the table's order
    place = s["count"].long() + torch.cumsum(back.reshape(-1), 0).view(n, width) - 1
    spare = torch.cat([pool, pool.new_zeros(1)])  # one entry past the end takes what is not kept
    spare[torch.where(back, place, pool.numel())] = tables
    pool.copy_(spare[:-1])
    avail = s["count"].long() + back.sum()
    held = torch.where(gone, 0, s["held"].long())
    total = (cached + runs + bs - 1) // bs
    fits = total <= width
    need = torch.where(fits & ~gone, (total - held).clamp(min=0), 0)
    cum = torch.cumsum(need, 0)
    given = ~gone & fits & ((need == 0) | (cum <= avail))
    need = torch.where(given, need, 0)
    fresh = (col >= held[:, None]) & (col < (held + need)[:, None])
    take = (avail - 1 - (cum - need)[:, None] - (col - held[:, None])).clamp(0, pool.numel() - 1)
    tables.copy_(torch.where(fresh, pool[take], tables))
    row = torch.searchsorted(cu[1:], torch.arange(t, device=cu.device), right=True)
    pos = cached[row] + torch.arange(t, device=cu.device) - cu[row]
    slot = tables[row, (pos // bs).clamp(max=width - 1)] * bs + pos % bs
    slot = torch.where(given[row], slot, -1)
    i32 = torch.int32
    return (torch.where(given, cached + runs, cached).to(i32), (held + need).to(i32),
            (avail - need.sum()).to(i32).view(1), pos.to(i32), slot.to(i32), tables, pool)


def _verify(s):
    p, q, tokens, cu = s["p"], s["q"], s["tokens"].long(), s["cu"].long()
    t, v = p.shape
    n = cu.numel() - 1
    runs = cu[1:] - cu[:-1]
    at = torch.arange(t, device=p.device)
    row = torch.searchsorted(cu[1:], at, right=True)
    i = at - cu[row]
    draft = torch.roll(tokens, -1)  # row i of a run judges its token i + 1
    px = p.gather(1, draft[:, None])[:, 0].float()
    qx = q.gather(1, draft[:, None])[:, 0].float() if q is not None else torch.ones_like(px)
    holds = s["u"] * qx < px
    ends = (i == runs[row] - 1) | ~holds  # the first such row of a run is where it stops
    stop = torch.full((n,), t, device=p.device).scatter_reduce_(
        0, row, torch.where(ends, at, t), "amin")
    live = runs > 0
    took = torch.where(live, stop - cu[:-1], 0)
    stop = stop.clamp(max=t - 1)
    w = p[stop].float()
    fell = live & (took < runs - 1)
    if q is not None:
        less = (w - q[stop].float()).clamp(min=0)
    else:
        less = w.scatter(1, draft[stop][:, None], 0.0)
    less = torch.where((less > 0).any(1, keepdim=True), less, w)
    w = torch.where(fell[:, None], less, w)
    race = torch.where(w > 0, w / s["e"], torch.zeros_like(w))
    best = race.amax(1, keepdim=True)
    token = torch.where(race == best, torch.arange(v, device=p.device), v).amin(1)
    token = torch.where(live, token, -1)
    out = torch.where(i < took[row], draft, torch.where(i == took[row], token[row], -1))
    i32 = torch.int32
    return torch.where(live, took + 1, 0).to(i32), token.to(i32), out.to(i32)


# ---------------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    if case["op"] == "attend":
        return _exact_attend(prepare(case, seed))
    if case["op"] == "append":
        return _exact_append(prepare(case, seed))
    return None  # the plan and the verdicts are whole numbers


def _exact_attend(s):
    """For each request and key head: softmax(q k^T / sqrt(D)) v over the keys a token may see."""
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    cu, ctx = s["cu"].tolist(), s["ctx"].tolist()
    kv, bs = s["kc"].shape[1:3]
    g = s["q"].shape[1] // kv
    for r in range(len(ctx)):
        pages = s["tables"][r, :-(-ctx[r] // bs)].long()
        n = cu[r + 1] - cu[r]
        hidden = torch.ones(n, ctx[r], dtype=torch.bool, device=DEV).triu(ctx[r] - n + 1)
        for j in range(kv):
            k, v = ((c[pages, j].double() * a[pages, j].double()[:, None, None]).flatten(0, 1)[:ctx[r]]
                    for c, a in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))
            for h in range(j * g, j * g + g):
                z = s["q"][cu[r]:cu[r + 1], h].double() @ k.T / math.sqrt(D)
                z.masked_fill_(hidden, -math.inf)
                out[cu[r]:cu[r + 1], h] = torch.softmax(z, -1) @ v
    return out


def _nearest(x):
    """The e4m3 number nearest to x, ties to even: three fraction bits, exponents from -6."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return torch.round(x / step) * step


def _exact_append(s):
    """Page after page: the scale from the largest of what is written and what was there."""
    bs, slots = s["kc"].shape[2], s["slots"].tolist()
    groups = []  # (first token, count) of the tokens that share a page
    for i, x in enumerate(slots):
        if groups and x // bs == slots[i - 1] // bs:
            groups[-1][1] += 1
        else:
            groups.append([i, 1])
    got = []
    for x, c, a in ((s["k"], s["kc"], s["ks"]), (s["v"], s["vc"], s["vs"])):
        x, c, a = x.double(), c.double(), a.double()
        for i, m in groups:
            page, off = slots[i] // bs, slots[i] % bs
            new = x[i:i + m].transpose(0, 1)  # [kv, m, D]
            scale = torch.exp2(torch.ceil(torch.log2(new.abs().amax((1, 2)) / 448)).clamp(min=-100))
            if off:
                scale = torch.maximum(scale, a[page])
                c[page, :, :off] = _nearest(c[page, :, :off] * (a[page] / scale)[:, None, None])
            a[page] = scale
            c[page, :, off:off + m] = _nearest(new / scale[:, None, None])
        got += [c, a]
    return got[0], got[2], got[1], got[3]
