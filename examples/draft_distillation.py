"""A draft model's output layer trained on what the target recorded while it served.

    python examples/draft_distillation.py [steps]

The target's logits are recorded as their largest entries' log probabilities (``token_logprobs``); the
draft's output layer is then trained towards them with ``distill_topk_grad``, which gives losses and the
gradient in the logits in one call.  Hidden states and weights are random tables.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import kimi_delta_attention_03_gb300 as kda  # noqa: E402

TOKENS, HIDDEN, VOCAB, ENTRIES = 256, 64, 4001, 24


def record(logits):
    """What a server keeps of the target's logits."""
    _, _, ids, logprobs = kda.token_logprobs(logits, top_k=ENTRIES)
    return ids, logprobs


def gradient(hidden, head, ids, logprobs, weight):
    """Losses of the draft's tokens and the gradient of their weighted sum in its output layer."""
    loss, d_logits = kda.distill_topk_grad(hidden @ head, ids, logprobs, weight, tail=True)
    return loss, hidden.T @ d_logits


def main(steps=20):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(0)
    randn = lambda *shape: torch.randn(*shape, generator=g, device=dev)  # noqa: E731
    hidden = randn(TOKENS, HIDDEN)
    target, head = randn(HIDDEN, VOCAB) * 0.4, randn(HIDDEN, VOCAB) * 0.4
    ids, logprobs = record(hidden @ target)
    weight = torch.full((TOKENS,), 1.0 / TOKENS, device=dev)
    for s in range(steps):
        loss, d_head = gradient(hidden, head, ids, logprobs, weight)
        head -= 20.0 * d_head
        print(f"step {s}: divergence {float(loss.mean()):.4f}")
    assert kda.read_device_status() == 0
    return loss


if __name__ == "__main__":
    main(*map(int, sys.argv[1:2]))
