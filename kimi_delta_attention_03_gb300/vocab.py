"""Operators over rows of vocabulary logits, next to draft verification: log probabilities of given
tokens with entropy and alternatives, and distillation from a teacher's top entries
(``include/kda.h``, "Vocabulary rows").

Argument marshalling only, like ``paged``; ``stream`` is treated as it is there.
"""
from __future__ import annotations

import torch
from torch import empty_like

from . import binding
from .binding import KDA_OK, KdaError, run_on
from .paged import _BF16, _F32, _I32, _check, _cuda, _lib, _stream

_MOST = 2 ** 31 - 1  # of the C ABI's int32 sizes, which ctypes would wrap; the library refuses it


def _rows(name, x, dev):
    """(T, V, row stride) of [T, V] logits whose rows may lie apart."""
    s = x.stride()
    if (x.dtype is not _BF16 and x.dtype is not _F32) or x.get_device() != dev or len(s) != 2 \
            or (s[1] != 1 and x.shape[1] > 1):
        raise ValueError(f"{name}: expected bf16 or fp32 [T, V] with contiguous rows on cuda:{dev}, "
                         f"got {x.dtype} {tuple(x.shape)} with strides {s} on {x.device}")
    t, v = x.shape
    return t, min(v, _MOST), s[0] if t > 1 else v


def token_logprobs(logits, tokens=None, top_k: int = 0, inv_temperature=None, stream=None):
    """Log probabilities of given tokens, the rows' entropies and their likeliest alternatives.

    logits: bf16 or fp32 [T, V], rows at any stride of V or more; tokens: int32 [T] or None (a negative
    token: the row is skipped); inv_temperature: fp32 [T], above 0 and at most 2^127, or None (ones).  Returns
    (logprobs [T] or None without tokens, entropy [T], top_ids [T, top_k], top_logprobs [T, top_k]); ids
    int32, the others fp32."""
    if stream is not None:
        return run_on(stream, token_logprobs, logits, tokens, top_k, inv_temperature)
    dev = _cuda("token_logprobs", logits)
    t, v, stride = _rows("logits", logits, dev)
    if tokens is not None:
        _check("tokens", tokens, (t,), _I32, dev)
    if inv_temperature is not None:
        _check("inv_temperature", inv_temperature, (t,), _F32, dev)
    if not 0 <= top_k <= 128:
        raise ValueError(f"top_k: expected 0 .. 128, got {top_k}")
    device = logits.device
    entropy = torch.empty(t, dtype=_F32, device=device)
    logprobs = None if tokens is None else empty_like(entropy)
    ids = torch.empty((t, top_k), dtype=_I32, device=device)
    best = torch.empty((t, top_k), dtype=_F32, device=device)
    st = _lib().kda_token_logprobs(
        t, v, binding._DTYPES[logits.dtype], logits.data_ptr(), stride,
        None if tokens is None else tokens.data_ptr(),
        None if inv_temperature is None else inv_temperature.data_ptr(), top_k,
        None if logprobs is None else logprobs.data_ptr(), entropy.data_ptr(),
        ids.data_ptr(), best.data_ptr(), _stream(None, dev))
    if st != KDA_OK:
        raise KdaError(st, "kda_token_logprobs")
    return logprobs, entropy, ids, best


def _teacher(ids, values, t, dev):
    if ids.dim() != 2:
        raise ValueError(f"teacher_ids: expected [T, K], got {tuple(ids.shape)}")
    k = ids.shape[1]
    _check("teacher_ids", ids, (t, k), _I32, dev)
    _check("teacher_values", values, (t, k), _F32, dev)
    return min(k, _MOST)


def _gradient(logits, d_logits, t, v, dev):
    if d_logits is None:
        d_logits = torch.empty((t, v), dtype=logits.dtype, device=logits.device)
    dt, dv, stride = _rows("d_logits", d_logits, dev)
    if (dt, dv) != (t, v) or d_logits.dtype is not logits.dtype:
        raise ValueError(f"d_logits: expected {logits.dtype} {(t, v)}, got {d_logits.dtype} {(dt, dv)}")
    return d_logits, stride


def distill_topk(logits, teacher_ids, teacher_values, inv_temperature: float = 1.0,
                 tail: bool = False, stream=None):
    """Kullback-Leibler divergence of softmax(logits * inv_temperature) from a teacher's top entries.

    logits: bf16 or fp32 [T, V], rows at any stride of V or more; teacher_ids: int32 [T, K] (negative: absent);
    teacher_values: fp32 [T, K], logits or log probabilities, of which the softmax is taken, or with
    ``tail`` log probabilities, and what they leave of 1 is the outcome of all other tokens.  Returns
    (loss [T], stats [T, 4]), fp32; ``distill_topk_bwd`` takes the stats."""
    if stream is not None:
        return run_on(stream, distill_topk, logits, teacher_ids, teacher_values, inv_temperature, tail)
    dev = _cuda("distill_topk", logits)
    t, v, stride = _rows("logits", logits, dev)
    k = _teacher(teacher_ids, teacher_values, t, dev)
    loss = torch.empty(t, dtype=_F32, device=logits.device)
    stats = torch.empty((t, 4), dtype=_F32, device=logits.device)
    st = _lib().kda_distill_topk(
        t, v, binding._DTYPES[logits.dtype], logits.data_ptr(), stride, k,
        teacher_ids.data_ptr(), teacher_values.data_ptr(), inv_temperature,
        1 if tail else 0, loss.data_ptr(), stats.data_ptr(), _stream(None, dev))
    if st != KDA_OK:
        raise KdaError(st, "kda_distill_topk")
    return loss, stats


def distill_topk_bwd(d_loss, logits, teacher_ids, teacher_values, stats,
                     inv_temperature: float = 1.0, tail: bool = False, d_logits=None, stream=None):
    """Gradient of ``distill_topk``'s losses in the logits, for their gradients d_loss, fp32 [T].

    stats: from ``distill_topk`` on the same inputs.  ``d_logits``: [T, V] of the logits' type, rows at
    any stride of V or more; it may be ``logits``, which is overwritten then, and must not overlap them
    otherwise.  Returns it."""
    if stream is not None:
        return run_on(stream, distill_topk_bwd, d_loss, logits, teacher_ids, teacher_values, stats,
                      inv_temperature, tail, d_logits)
    dev = _cuda("distill_topk_bwd", logits)
    t, v, stride = _rows("logits", logits, dev)
    k = _teacher(teacher_ids, teacher_values, t, dev)
    _check("d_loss", d_loss, (t,), _F32, dev)
    _check("stats", stats, (t, 4), _F32, dev)
    d_logits, d_stride = _gradient(logits, d_logits, t, v, dev)
    st = _lib().kda_distill_topk_bwd(
        t, v, binding._DTYPES[logits.dtype], logits.data_ptr(), stride, k,
        teacher_ids.data_ptr(), teacher_values.data_ptr(), inv_temperature,
        1 if tail else 0, stats.data_ptr(), d_loss.data_ptr(),
        d_logits.data_ptr(), d_stride, _stream(None, dev))
    if st != KDA_OK:
        raise KdaError(st, "kda_distill_topk_bwd")
    return d_logits


def distill_topk_grad(logits, teacher_ids, teacher_values, weight, inv_temperature: float = 1.0,
                      tail: bool = False, d_logits=None, stream=None):
    """``distill_topk``'s losses and the gradient of sum(weight * loss) in one launch, which reads the
    logits a second time while L2 has them.

    weight: fp32 [T]; the others as for ``distill_topk`` and ``distill_topk_bwd``.  Returns (loss [T],
    unweighted, d_logits)."""
    if stream is not None:
        return run_on(stream, distill_topk_grad, logits, teacher_ids, teacher_values, weight,
                      inv_temperature, tail, d_logits)
    dev = _cuda("distill_topk_grad", logits)
    t, v, stride = _rows("logits", logits, dev)
    k = _teacher(teacher_ids, teacher_values, t, dev)
    _check("weight", weight, (t,), _F32, dev)
    d_logits, d_stride = _gradient(logits, d_logits, t, v, dev)
    loss = torch.empty(t, dtype=_F32, device=logits.device)
    st = _lib().kda_distill_topk_grad(
        t, v, binding._DTYPES[logits.dtype], logits.data_ptr(), stride, k,
        teacher_ids.data_ptr(), teacher_values.data_ptr(), inv_temperature,
        1 if tail else 0, weight.data_ptr(), loss.data_ptr(),
        d_logits.data_ptr(), d_stride, _stream(None, dev))
    if st != KDA_OK:
        raise KdaError(st, "kda_distill_topk_grad")
    return loss, d_logits
