"""Plain host implementations of the paged serving operators, one loop per definition, in 64 bits
(whole numbers and the fp32 comparisons of the draft verification exactly)."""
from __future__ import annotations

import numpy as np
import torch

E4M3 = torch.float8_e4m3fn


def plan(cached, cu, tables, held, free, count, bs, t, release=None):
    """Returns (context, held, free_count, positions, slots, tables, free list)."""
    tables, free = [list(r) for r in tables], list(free)
    n, width = len(cached), len(tables[0]) if tables else 0
    release = [0] * n if release is None else release
    for i in range(n):
        if release[i]:
            for page in tables[i][:held[i]]:
                free[count] = page
                count += 1
    demand, taken = 0, 0
    context, kept, positions, slots = [], [], [0] * t, [-1] * t
    for i in range(n):
        run, c = cu[i + 1] - cu[i], 0 if release[i] else cached[i]
        have = 0 if release[i] else held[i]
        total = -(-(c + run) // bs)
        served = not release[i] and total <= width
        need = max(0, total - have) if served else 0
        demand += need
        served = served and (need == 0 or demand <= count)
        if served:
            for j in range(need):
                tables[i][have + j] = free[count - 1 - taken]
                taken += 1
            have += need
        context.append(c + run if served else c)
        kept.append(have)
        for k in range(run):
            pos = c + k
            positions[cu[i] + k] = pos
            if served:
                slots[cu[i] + k] = tables[i][pos // bs] * bs + pos % bs
    return context, kept, count - taken, positions, slots, tables, free


def nearest_e4m3(x):
    """The e4m3 number nearest to x (|x| <= 464), ties to even: 3 fraction bits, exponents >= -6."""
    x = np.asarray(x, dtype=np.float64)
    _, e = np.frexp(x)
    step = np.exp2(np.maximum(e - 1, -6).astype(np.float64) - 3)
    return np.round(x / step) * step


def scale_for(amax):
    if amax == 0:
        return 2.0 ** -100
    e = -100
    while amax > 448 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append(x, slots, codes, scale):
    """x [T, H, 128], codes [pages, H, bs, 128] (values), scale [pages, H]: float64 arrays, codes and
    scale updated in place."""
    bs = codes.shape[2]
    t = 0
    while t < len(slots):
        if slots[t] < 0:
            t += 1
            continue
        page, m = slots[t] // bs, 1
        while t + m < len(slots) and slots[t + m] >= 0 and slots[t + m] // bs == page:
            m += 1
        first = slots[t] % bs
        for h in range(x.shape[1]):
            new = x[t:t + m, h]
            s = scale_for(np.abs(new[np.isfinite(new)]).max(initial=0.0))
            if first:
                old = scale[page, h]
                s = max(s, old)
                if s > old:
                    codes[page, h, :first] = nearest_e4m3(codes[page, h, :first] * (old / s))
            scale[page, h] = s
            for i in range(m):
                y = new[i] / s
                codes[page, h, slots[t + i] % bs] = np.where(np.isfinite(y), nearest_e4m3(
                    np.where(np.isfinite(y), y, 0)), np.nan)
        t += m


def attention(q, cu, tables, ctx, kc, vc, ks, vs, sm_scale=128 ** -0.5):
    """All tensors on the host.  Returns (out, spread, top, most): float64 [T, H, 128] outputs, the
    weighted mean of |v|, the largest |q| |k| scale of each row, and the sum of |v| over the keys
    it sees (for error bounds)."""
    t, h, d = q.shape
    kv, bs = kc.shape[1], kc.shape[2]
    g = h // kv
    out = np.zeros((t, h, d))
    spread = np.zeros((t, h, d))
    top = np.zeros((t, h, 1))
    most = np.zeros((t, h, d))
    qd, kc, vc = q.double().numpy(), kc.double(), vc.double()
    for n in range(len(ctx)):
        run = cu[n + 1] - cu[n]
        if run == 0 or ctx[n] <= 0:
            continue
        pages = torch.as_tensor(tables[n][:-(-ctx[n] // bs)]).long()
        for j in range(kv):
            k = (kc[pages, j] * ks[pages, j].double()[:, None, None]).reshape(-1, d)[:ctx[n]].numpy()
            v = (vc[pages, j] * vs[pages, j].double()[:, None, None]).reshape(-1, d)[:ctx[n]].numpy()
            for i in range(run):
                keys = ctx[n] - run + i + 1
                if keys <= 0:
                    continue
                x = qd[cu[n] + i, j * g:(j + 1) * g]
                z = x @ k[:keys].T * sm_scale
                w = np.exp(z - z.max(1, keepdims=True))
                w /= w.sum(1, keepdims=True)
                out[cu[n] + i, j * g:(j + 1) * g] = w @ v[:keys]
                spread[cu[n] + i, j * g:(j + 1) * g] = w @ np.abs(v[:keys])
                most[cu[n] + i, j * g:(j + 1) * g] = np.abs(v[:keys]).sum(0)
                top[cu[n] + i, j * g:(j + 1) * g, 0] = (np.abs(x) @ np.abs(k[:keys]).T * sm_scale).max(1)
    return out, spread, top, most


def verify(p, q, tokens, cu, u, e):
    """fp32 arrays; q may be None.  Returns (commit, next_token, out_tokens)."""
    commit, nxt, out = [], [], [-1] * len(tokens)
    f = np.float32
    for n in range(len(cu) - 1):
        a, run = cu[n], cu[n + 1] - cu[n]
        if run == 0:
            commit.append(0)
            nxt.append(-1)
            continue
        took = 0
        while took < run - 1:
            x = tokens[a + took + 1]
            if not 0 <= x < p.shape[1]:
                break
            qx = f(1) if q is None else q[a + took, x]
            if not f(u[a + took] * qx) < p[a + took, x]:
                break
            took += 1
        w = p[a + took]
        if took < run - 1:
            x = tokens[a + took + 1]
            if q is None:
                less = w.copy()
                if 0 <= x < len(less):
                    less[x] = 0
            else:
                less = np.maximum(w - q[a + took], f(0))
            w = less if (less > 0).any() else w
        with np.errstate(divide="ignore", invalid="ignore"):
            race = np.where(w > 0, w / e[n], f(0)).astype(f)
        token = int(np.argmax(race))
        commit.append(took + 1)
        nxt.append(token)
        for i in range(took):
            out[a + i] = int(tokens[a + i + 1])
        out[a + took] = token
    return commit, nxt, out
