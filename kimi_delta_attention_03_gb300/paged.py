"""Paged serving of the layers next to KDA: page plan, 8-bit cache append, paged attention and
draft verification (``include/kda.h``, "Paged serving").

Argument marshalling only, like ``binding``.  The kernels take some microseconds, no longer than
the host needs for a call, so the checks are a few attribute reads each, and results are allocated
one by one (1.5 us each; splitting one allocation takes longer).

``stream``: the kernels run there, and what the call allocates is that stream's memory.  What the
caller passes in has to be ready there and to stay until the kernels are done (``record_stream`` or
an event, where it is another stream's memory); so have the results before another stream reads them.
Tensors on another device than the current one are refused, as the kernels run on that; where a call
allocates, a given stream's device is the current one.
"""
from __future__ import annotations

import torch
from torch import empty_like

from . import binding
from .binding import KDA_OK, KdaError, run_on

_BF16, _F32, _I32, _E4M3 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn
_D = 128


def _lib():
    return binding._lib or binding.load_library()


def _stream(stream, dev):
    """Handle of the given stream, or of the current one of device index ``dev`` (without the
    Stream object that torch.cuda.current_stream builds, which costs 2 us)."""
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _check(name, t, shape, dtype, dev):
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {dtype} {tuple(shape)} on cuda:{dev}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")


def _rows(name, t, heads, dev):
    """The token stride of a [T, heads, 128] bf16 tensor whose tokens may lie apart."""
    s = t.stride()
    if (t.dtype is not _BF16 or t.get_device() != dev or len(s) != 3 or t.shape[1] != heads
            or t.shape[2] != _D or s[2] != 1 or (s[1] != _D and heads > 1)):
        raise ValueError(f"{name}: expected bf16 [T, {heads}, {_D}] with contiguous heads on "
                         f"cuda:{dev}, got {t.dtype} {tuple(t.shape)} with strides {s} on {t.device}")
    return s[0] if t.shape[0] > 1 else heads * _D


def _cache(k_cache, v_cache, k_scale, v_scale, dev):
    shape = k_cache.shape
    if len(shape) != 4 or shape[3] != _D:
        raise ValueError(f"k_cache: expected [pages, heads, page_size, {_D}], got {tuple(shape)}")
    _check("k_cache", k_cache, shape, _E4M3, dev)
    _check("v_cache", v_cache, shape, _E4M3, dev)
    _check("k_scale", k_scale, shape[:2], _F32, dev)
    _check("v_scale", v_scale, shape[:2], _F32, dev)
    return shape[0], shape[1], shape[2]


def _cuda(name, t):
    if not t.is_cuda:
        raise ValueError(f"{name} needs CUDA tensors")
    dev = t.get_device()
    if dev != torch._C._cuda_getDevice():  # where the kernels run (torch.cuda.current_device takes twice the 0.12 us)
        raise ValueError(f"{name}: tensors on cuda:{dev}, which is not the current device")
    return dev


def paged_plan(cached_lens, cu_seqlens, block_tables, held, free_list, free_count, page_size: int,
               total_tokens: int, release=None, stream=None):
    """Block tables, positions and cache slots of a step from device lengths.

    cached_lens, held, release (or None): int32 [N]; cu_seqlens: int32 [N+1], the runs' offsets;
    block_tables: int32 [N, width], new pages are written in place; free_list: int32 [capacity],
    free_count: int32 [1] entries in use, released pages are written after them; total_tokens:
    rows of the two per-token results.  Returns (context_lens [N], held [N], free_count [1],
    positions [T], slot_map [T]), int32; a token without a page has slot -1."""
    if stream is not None:
        return run_on(stream, paged_plan, cached_lens, cu_seqlens, block_tables, held, free_list,
                      free_count, page_size, total_tokens, release)
    dev = _cuda("paged_plan", cached_lens)
    n, width = block_tables.shape
    t = int(total_tokens)
    _check("cached_lens", cached_lens, (n,), _I32, dev)
    _check("cu_seqlens", cu_seqlens, (n + 1,), _I32, dev)
    _check("block_tables", block_tables, (n, width), _I32, dev)
    _check("held", held, (n,), _I32, dev)
    capacity = free_list.numel()
    _check("free_list", free_list, (capacity,), _I32, dev)
    _check("free_count", free_count, (1,), _I32, dev)
    if release is not None:
        _check("release", release, (n,), _I32, dev)
    if t < 0:
        raise ValueError("total_tokens must not be negative")
    context, kept, left = empty_like(cached_lens), empty_like(cached_lens), empty_like(free_count)
    positions = torch.empty(t, dtype=_I32, device=cached_lens.device)
    slots = empty_like(positions)
    st = _lib().kda_paged_plan(
        n, width, page_size, t, capacity, cached_lens.data_ptr(), cu_seqlens.data_ptr(),
        None if release is None else release.data_ptr(), held.data_ptr(),
        block_tables.data_ptr() or None, free_list.data_ptr() or None, free_count.data_ptr(),
        context.data_ptr(), kept.data_ptr(), left.data_ptr(), positions.data_ptr() or None,
        slots.data_ptr() or None, _stream(None, dev))
    if st != KDA_OK:
        raise KdaError(st, "kda_paged_plan")
    return context, kept, left, positions, slots


def paged_append(k, v, slot_map, k_cache, v_cache, k_scale, v_scale, stream=None):
    """Write the tokens' keys and values into their cache slots, coded in e4m3.

    k, v: bf16 [T, Hkv, 128], tokens at any stride (slices of a fused projection); slot_map: int32
    [T] (negative: not written).  k_cache, v_cache: float8_e4m3fn [pages, Hkv, page_size, 128] and
    k_scale, v_scale: fp32 [pages, Hkv], updated in place."""
    dev = _cuda("paged_append", k)
    pages, heads, bs = _cache(k_cache, v_cache, k_scale, v_scale, dev)
    t = k.shape[0]
    ks, vs = _rows("k", k, heads, dev), _rows("v", v, heads, dev)
    if v.shape[0] != t:
        raise ValueError(f"v: expected {t} tokens, got {v.shape[0]}")
    _check("slot_map", slot_map, (t,), _I32, dev)
    st = _lib().kda_paged_append(t, heads, bs, pages, k.data_ptr(), ks, v.data_ptr(), vs,
                                 slot_map.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                 k_scale.data_ptr(), v_scale.data_ptr(), _stream(stream, dev))
    if st != KDA_OK:
        raise KdaError(st, "kda_paged_append")


def paged_attention_workspace_bytes(num_heads: int, num_kv_heads: int, max_run: int) -> int:
    return _lib().kda_paged_attention_workspace_bytes(num_heads, num_kv_heads, max_run)


def paged_attention(q, cu_seqlens, block_tables, context_lens, k_cache, v_cache, k_scale, v_scale,
                    max_run: int, sm_scale: float = _D ** -0.5, out=None, workspace=None,
                    stream=None):
    """Attention of every run token over its request's pages (causal within the run).

    q: bf16 [T, H, 128], tokens at any stride; cu_seqlens: int32 [N+1]; block_tables: int32 [N,
    width]; context_lens: int32 [N], the run included; the cache as for ``paged_append``; max_run:
    the longest run.  ``workspace``: a uint8 tensor of paged_attention_workspace_bytes(...) bytes;
    allocated when not given.  Returns out, bf16 [T, H, 128]."""
    if stream is not None:
        return run_on(stream, paged_attention, q, cu_seqlens, block_tables, context_lens, k_cache,
                      v_cache, k_scale, v_scale, max_run, sm_scale, out, workspace)
    dev = _cuda("paged_attention", q)
    pages, kv, bs = _cache(k_cache, v_cache, k_scale, v_scale, dev)
    t, h = q.shape[0], q.shape[1]
    stride = _rows("q", q, h, dev)
    n, width = block_tables.shape
    _check("cu_seqlens", cu_seqlens, (n + 1,), _I32, dev)
    _check("block_tables", block_tables, (n, width), _I32, dev)
    _check("context_lens", context_lens, (n,), _I32, dev)
    if out is None:
        out = torch.empty((t, h, _D), dtype=_BF16, device=q.device)
    else:
        _check("out", out, (t, h, _D), _BF16, dev)
    lib = _lib()
    need = lib.kda_paged_attention_workspace_bytes(h, kv, max_run)
    if workspace is None:
        ws, size = torch.empty(need, dtype=torch.uint8, device=q.device), need
    else:
        ws, size = workspace, workspace.numel() * workspace.element_size()
        if ws.get_device() != dev or not ws.is_contiguous():
            raise ValueError(f"workspace: expected a contiguous tensor on cuda:{dev}")
    st = lib.kda_paged_attention(
        n, t, h, kv, bs, pages, width, max_run, sm_scale, q.data_ptr(), stride,
        cu_seqlens.data_ptr(), block_tables.data_ptr() or None, context_lens.data_ptr(),
        k_cache.data_ptr() or None, v_cache.data_ptr() or None, k_scale.data_ptr() or None,
        v_scale.data_ptr() or None, out.data_ptr(), ws.data_ptr(), size,
        _stream(None, dev))
    if st != KDA_OK:
        raise KdaError(st, "kda_paged_attention")
    return out


def verify_draft(target_probs, tokens, cu_seqlens, uniform, noise, draft_probs=None, stream=None):
    """Which drafted tokens hold and the token after them, from given random numbers.

    target_probs, draft_probs (or None: certain drafts): [T, V] fp32 or bf16; tokens: int32 [T], per
    run the last token and its drafts; cu_seqlens: int32 [N+1]; uniform: fp32 [T] in [0, 1); noise:
    fp32 [N, V], exponentially distributed.  Returns (commit [N], next_token [N], out_tokens [T]),
    int32: commit is what ``decode_window`` takes, out_tokens each run's accepted drafts and next
    token, then -1."""
    if stream is not None:
        return run_on(stream, verify_draft, target_probs, tokens, cu_seqlens, uniform, noise, draft_probs)
    dev = _cuda("verify_draft", target_probs)
    t, v = target_probs.shape
    n = cu_seqlens.numel() - 1
    dt = target_probs.dtype
    _check("target_probs", target_probs, (t, v), dt, dev)
    if draft_probs is not None:
        _check("draft_probs", draft_probs, (t, v), dt, dev)
    _check("tokens", tokens, (t,), _I32, dev)
    _check("cu_seqlens", cu_seqlens, (n + 1,), _I32, dev)
    _check("uniform", uniform, (t,), _F32, dev)
    _check("noise", noise, (n, v), _F32, dev)
    commit = torch.empty(n, dtype=_I32, device=tokens.device)
    token, out = empty_like(commit), empty_like(tokens)
    st = _lib().kda_verify_draft(
        n, t, v, binding._DTYPES.get(dt, 99), target_probs.data_ptr() or None,
        None if draft_probs is None else draft_probs.data_ptr() or None, tokens.data_ptr() or None,
        cu_seqlens.data_ptr(), uniform.data_ptr() or None, noise.data_ptr(), commit.data_ptr(),
        token.data_ptr(), out.data_ptr() or None, _stream(None, dev))
    if st != KDA_OK:
        raise KdaError(st, "kda_verify_draft")
    return commit, token, out
