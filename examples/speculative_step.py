"""Speculative decoding of a small hybrid: one KDA layer and one full-attention layer share a step.

    python examples/speculative_step.py [steps]

Every request's run of a step is its last token and some drafts.  The step plans pages for the run,
writes the run's keys and values into the 8-bit cache, attends over it, runs the KDA window without
moving its state, verifies the drafts against the target's probabilities and then moves the state by
the tokens that stand.  The "model" is synthetic: projections are rows of random tables, one for
each token of the vocabulary, and the drafts come from a random table of token pairs.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import kimi_delta_attention_03_gb300 as kda  # noqa: E402

HEADS, KV_HEADS, D, VOCAB, PAGE = 8, 2, 128, 997, 16
I32, BF16 = torch.int32, torch.bfloat16


class Model:
    """Random tables in place of weights."""

    def __init__(self, device, seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        randn = lambda *shape: torch.randn(*shape, generator=g, device=device)  # noqa: E731
        unit = lambda x: torch.nn.functional.normalize(x, dim=-1)               # noqa: E731
        self.qkv = randn(VOCAB, HEADS + 2 * KV_HEADS, D).to(BF16)
        self.kda_q = (unit(randn(VOCAB, HEADS, D)) * D ** -0.5).to(BF16)
        self.kda_k, self.kda_v = unit(randn(VOCAB, HEADS, D)).to(BF16), randn(VOCAB, HEADS, D).to(BF16)
        self.log_alpha = (-0.1 * torch.rand(VOCAB, HEADS, D, generator=g, device=device)).to(BF16)
        self.beta = torch.rand(VOCAB, HEADS, generator=g, device=device).to(BF16)
        self.head = randn(2 * HEADS * D, VOCAB) * (2 * HEADS * D) ** -0.5 * 4
        self.pairs = torch.softmax(randn(VOCAB, VOCAB), -1)

    def kda_inputs(self, tokens):
        t = tokens.long()
        return self.kda_q[t], self.kda_k[t], self.kda_v[t], self.log_alpha[t], self.beta[t]


class Requests:
    """What a server keeps between steps, all of it on the device."""

    def __init__(self, first_tokens, pages, width, device):
        n = len(first_tokens)
        self.last = torch.tensor(first_tokens, dtype=I32, device=device)
        self.cached = torch.zeros(n, dtype=I32, device=device)
        self.held = torch.zeros(n, dtype=I32, device=device)
        self.tables = torch.full((n, width), -1, dtype=I32, device=device)
        self.free = torch.arange(pages, dtype=I32, device=device)
        self.count = torch.tensor([pages], dtype=I32, device=device)
        shape = (pages, KV_HEADS, PAGE, D)
        self.kc, self.vc = (torch.zeros(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
                            for _ in "kv")
        self.ks, self.vs = (torch.ones(pages, KV_HEADS, device=device) for _ in "kv")
        self.state = torch.zeros(n, HEADS, D, D, device=device)


def step(model, req, drafts, gen):
    """One step with `drafts` drafts a request.  Returns (out_tokens [N, drafts + 1], commit [N])."""
    n, run, dev = len(req.last), drafts + 1, req.last.device
    tokens = torch.empty(n, run, dtype=I32, device=dev)
    tokens[:, 0] = req.last
    draft_probs = torch.zeros(n, run, VOCAB, device=dev)
    for i in range(drafts):
        draft_probs[:, i] = model.pairs[tokens[:, i].long()]
        tokens[:, i + 1] = torch.multinomial(draft_probs[:, i], 1, generator=gen)[:, 0].to(I32)
    tokens, t = tokens.view(-1), n * run
    cu = (run * torch.arange(n + 1, device=dev)).to(I32)

    # full attention: pages, keys and values, attention
    context, req.held, req.count, positions, slots = kda.paged_plan(
        req.cached, cu, req.tables, req.held, req.free, req.count, PAGE, t)
    qkv = model.qkv[tokens.long()]  # a layer with positions would rotate by `positions` here
    q, k, v = qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV_HEADS], qkv[:, HEADS + KV_HEADS:]
    kda.paged_append(k, v, slots, req.kc, req.vc, req.ks, req.vs)
    full = kda.paged_attention(q, cu, req.tables, context, req.kc, req.vc, req.ks, req.vs, run)

    # KDA: the run's outputs, the state where it was
    nothing = torch.zeros(n, dtype=I32, device=dev)
    x, lens = model.kda_inputs(tokens), [run] * n
    linear = kda.decode_window(*x, cu, lens, req.state, commit=nothing)

    hidden = torch.cat([full.view(t, -1), linear.view(t, -1)], -1).float()
    target = torch.softmax(hidden @ model.head, -1)
    u = torch.rand(t, generator=gen, device=dev)
    noise = torch.empty(n, VOCAB, device=dev).exponential_(generator=gen)
    commit, req.last, out = kda.verify_draft(target, tokens, cu, u, noise,
                                             draft_probs=draft_probs.view(t, VOCAB))
    # the tokens that stand: into the KDA state, and so many of the cache
    kda.decode_window(*x, cu, lens, req.state, commit=commit, want_out=False)
    req.cached = req.cached + commit
    return out.view(n, run), commit, tokens.view(n, run)


def main(steps=8):
    dev, first = torch.device("cuda"), [3, 141, 59, 26, 535]
    model, req = Model(dev), Requests(first, pages=64, width=16, device=dev)
    gen = torch.Generator(device=dev).manual_seed(1)
    stood = [[] for _ in first]  # the tokens behind each request's state
    for s in range(steps):
        out, commit, tokens = step(model, req, drafts=s % 4, gen=gen)
        for r, c in enumerate(commit.tolist()):
            stood[r] += tokens[r, :c].tolist()
        print(f"step {s}: tokens kept {commit.tolist()}, next {req.last.tolist()}")
    assert req.cached.tolist() == [len(x) for x in stood]
    # the states are those of the kept tokens run one after another
    lens = [len(x) for x in stood]
    flat = torch.tensor(sum(stood, []), dtype=I32, device=dev)
    cu = torch.tensor([0] + lens, device=dev).cumsum(0).to(I32)
    state = torch.zeros_like(req.state)
    kda.decode_window(*model.kda_inputs(flat), cu, lens, state, want_out=False)
    assert torch.equal(state, req.state), "states"
    assert kda.read_device_status() == 0
    print("states match the kept tokens")


if __name__ == "__main__":
    main(*map(int, sys.argv[1:2]))
