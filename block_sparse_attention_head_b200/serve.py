"""Binding of the language-model entry points of ``libinstagen.so``:
``prompt_attention``, ``key_weights``, ``prefix_attention`` and ``evict``
(argument marshalling only; the contracts are in ``include/instagen.h``)."""
from __future__ import annotations

import ctypes
import math
from typing import Optional

import torch

from . import CacheParams, InstaGenError, PromptParams, _check, _need, _ptr, _stream, lib

_DTYPES = {torch.bfloat16: 0, torch.float16: 1}  # instagen_dtype


def _on_current(*tensors):
    """Kernels run on the current device, so every tensor must live there."""
    cur = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != cur:
            raise InstaGenError(f"tensors must be on the current device cuda:{cur}, got {t.device}")


def _dtype_of(t, name: str):
    if not isinstance(t, torch.Tensor) or t.dtype not in _DTYPES:
        raise TypeError(f"{name} must be a bfloat16 or float16 torch.Tensor")
    return t.dtype


def _need_rows(t, name: str, dtype, shape):
    """A 3-D tensor of rows: last dimension contiguous, the others strided in
    whole 16-byte steps without overlap."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise InstaGenError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    n0, n1, d = shape
    s0, s1, s2 = t.stride()
    if s2 != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    if (n0 > 1 and (s0 < d or s0 % 8)) or (n1 > 1 and (s1 < d or s1 % 8)):
        raise ValueError(f"{name}: strides must be multiples of 8 elements and at least a row, got {t.stride()}")


def _cache_shape(t, name: str, dtype):
    _need(t, name, dtype)
    if t.dim() != 4:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected [B, Hkv, slots, d]")
    return t.shape


def _work_area(workspace: Optional[torch.Tensor], need: int, like: torch.Tensor, what: str):
    if need == 0:
        raise InstaGenError(f"invalid or unsupported parameters for {what}")
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=like.device), need
    have = workspace.numel() * workspace.element_size()
    if have < need:
        raise InstaGenError(f"workspace too small: {have} < {need}")
    _on_current(workspace)
    return workspace, have


def _prompt_params(q, k, v, o, cu_q, cu_k, causal, softmax_scale) -> PromptParams:
    dt = _dtype_of(q, "q")
    if not isinstance(k, torch.Tensor):
        raise TypeError("k must be a torch.Tensor")
    if q.dim() != 3 or k.dim() != 3 or k.shape[2] != q.shape[2]:
        raise ValueError(f"q {tuple(q.shape)} and k {tuple(k.shape)} must be [Tq, Hq, d] and [Tk, Hkv, d]")
    Tq, Hq, d = q.shape
    Tk, Hkv = k.shape[:2]
    _need_rows(q, "q", dt, q.shape)
    _need_rows(k, "k", dt, k.shape)
    if Hkv < 1 or Hq < 1 or Hq % Hkv:
        raise ValueError(f"{Hq} query heads cannot share {Hkv} key/value heads")
    if v is not None:
        _need_rows(v, "v", dt, k.shape)
    if o is not None:
        _need_rows(o, "out", dt, q.shape)
    _need(cu_q, "cu_q", torch.int32)
    _need(cu_k, "cu_k", torch.int32, cu_q.shape)
    if cu_q.dim() != 1 or cu_q.numel() < 2:
        raise ValueError("cu_q must hold the starts of the sequences and the end of the last one")
    qs, ks = q.stride(), k.stride()
    vs, os = ks if v is None else v.stride(), qs if o is None else o.stride()
    return PromptParams(cu_q.numel() - 1, Hq, Hkv, d, Tq, Tk, _DTYPES[dt], 1 if causal else 0,
                        1.0 / math.sqrt(d) if softmax_scale is None else softmax_scale,
                        qs[0], qs[1], ks[0], ks[1], vs[0], vs[1], os[0], os[1])


def prompt_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_q: torch.Tensor, cu_k: torch.Tensor, *,
                     causal: bool = True, softmax_scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                     lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """Attention over packed prompts (instagen_prompt_attention): q [Tq, Hq, d],
    k and v [Tk, Hkv, d] bf16 or fp16 (views with 16-byte strides are read in
    place), cu_q and cu_k int32 [sequences + 1].  Query i of a sequence sees its
    keys j <= i + n_k - n_q (causal) or all of them.  Returns (O [Tq, Hq, d], lse
    [Hq, Tq] fp32); a row without keys is 0 with lse -inf.  Rows that belong to
    no sequence are not written (undefined unless ``out`` and ``lse`` are given)."""
    if not isinstance(v, torch.Tensor):
        raise TypeError("v must be a torch.Tensor")
    O = torch.empty(q.shape, dtype=q.dtype, device=q.device) if out is None and isinstance(q, torch.Tensor) else out
    p = _prompt_params(q, k, v, O, cu_q, cu_k, causal, softmax_scale)
    if lse is None:
        lse = torch.empty((p.Hq, p.Tq), dtype=torch.float32, device=q.device)
    else:
        _need(lse, "lse", torch.float32, (p.Hq, p.Tq))
    _on_current(q, k, v, cu_q, cu_k, O, lse)
    L, ref = lib(), ctypes.byref(p)
    ws, nws = _work_area(workspace, L.instagen_prompt_attention_workspace_size(ref), q, "instagen_prompt_attention")
    _check(L.instagen_prompt_attention(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_q), _ptr(cu_k), ref, _ptr(O), _ptr(lse),
                                       _ptr(ws), nws, _stream()), "instagen_prompt_attention")
    return O, lse


def key_weights(q: torch.Tensor, k: torch.Tensor, lse: torch.Tensor, cu_q: torch.Tensor, cu_k: torch.Tensor,
                weights: torch.Tensor, *, causal: bool = True, softmax_scale: Optional[float] = None,
                workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Adds to weights [Hkv, Tk] fp32 what every key gets of the queries'
    attention, summed over the queries that see it and the heads that share it
    (instagen_key_weights).  lse [Hq, Tq]: as ``prompt_attention`` returned it
    for these queries.  Returns weights."""
    p = _prompt_params(q, k, None, None, cu_q, cu_k, causal, softmax_scale)
    _need(lse, "lse", torch.float32, (p.Hq, p.Tq))
    _need(weights, "weights", torch.float32, (p.Hkv, p.Tk))
    _on_current(q, k, lse, cu_q, cu_k, weights)
    L, ref = lib(), ctypes.byref(p)
    ws, nws = _work_area(workspace, L.instagen_key_weights_workspace_size(ref), q, "instagen_key_weights")
    _check(L.instagen_key_weights(_ptr(q), _ptr(k), _ptr(lse), _ptr(cu_q), _ptr(cu_k), ref, _ptr(weights), _ptr(ws),
                                  nws, _stream()), "instagen_key_weights")
    return weights


def prefix_attention(q: torch.Tensor, k_prefix: Optional[torch.Tensor], v_prefix: Optional[torch.Tensor],
                     k_cache: torch.Tensor, v_cache: torch.Tensor, lens: torch.Tensor, *,
                     weights: Optional[torch.Tensor] = None, softmax_scale: Optional[float] = None,
                     out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None):
    """Attention of one token per sequence (instagen_prefix_attention): q [B, Hq,
    d] over the keys that the batch shares, k_prefix and v_prefix [Hkv, P, d]
    (None: none), and each sequence's own, k_cache and v_cache [B, Hkv, cap, d]
    of which lens [B] int32 are live.  With weights [B, Hkv, cap] fp32 the
    token's attention weights on its own keys are added to them.  Returns
    (O [B, Hq, d], lse [B, Hq] fp32)."""
    dt = _dtype_of(q, "q")
    B, Hkv, cap, d = _cache_shape(k_cache, "k_cache", dt)
    _need(v_cache, "v_cache", dt, k_cache.shape)
    if q.dim() != 3 or q.shape[0] != B or q.shape[2] != d:
        raise ValueError(f"q has shape {tuple(q.shape)}, expected ({B}, Hq, {d})")
    _need_rows(q, "q", dt, q.shape)
    Hq = q.shape[1]
    if Hq > 1 and q.stride(1) != d:
        raise ValueError("q: the heads of a token must be contiguous")
    if Hkv < 1 or Hq < 1 or Hq % Hkv:
        raise ValueError(f"{Hq} query heads cannot share {Hkv} key/value heads")
    if (k_prefix is None) != (v_prefix is None):
        raise ValueError("k_prefix and v_prefix come together")
    P, ph = 0, 0
    if k_prefix is not None:
        if not isinstance(k_prefix, torch.Tensor) or k_prefix.dim() != 3:
            raise ValueError("k_prefix must be a tensor [Hkv, P, d]")
        P = k_prefix.shape[1]
        _need_rows(k_prefix, "k_prefix", dt, (Hkv, P, d))
        _need_rows(v_prefix, "v_prefix", dt, (Hkv, P, d))
        ph = k_prefix.stride(0)
        if P > 1 and (k_prefix.stride(1) != d or v_prefix.stride(1) != d):
            raise ValueError("k_prefix, v_prefix: the rows of a head must be contiguous")
        if Hkv > 1 and P > 0 and v_prefix.stride(0) != ph:
            raise ValueError("k_prefix and v_prefix must have the same strides")
    _need(lens, "lens", torch.int32, (B,))
    if weights is not None:
        _need(weights, "weights", torch.float32, (B, Hkv, cap))
    if out is None:
        out = torch.empty((B, Hq, d), dtype=dt, device=q.device)
    else:
        _need(out, "out", dt, (B, Hq, d))
    if lse is None:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    else:
        _need(lse, "lse", torch.float32, (B, Hq))
    _on_current(q, k_prefix, v_prefix, k_cache, v_cache, lens, weights, out, lse)
    p = CacheParams(B, Hq, Hkv, d, P, cap, _DTYPES[dt], 1.0 / math.sqrt(d) if softmax_scale is None else softmax_scale,
                    q.stride(0), ph)
    L, ref = lib(), ctypes.byref(p)
    ws, nws = _work_area(workspace, L.instagen_prefix_attention_workspace_size(ref, weights is not None), q,
                         "instagen_prefix_attention")
    _check(L.instagen_prefix_attention(_ptr(q), _ptr(k_prefix), _ptr(v_prefix), _ptr(k_cache), _ptr(v_cache),
                                       _ptr(lens), ref, _ptr(out), _ptr(lse), _ptr(weights), _ptr(ws), nws,
                                       _stream()), "instagen_prefix_attention")
    return out, lse


def evict(k_cache: torch.Tensor, v_cache: torch.Tensor, weights: torch.Tensor, pos: torch.Tensor, lens: torch.Tensor,
          budget: int, recent: int, *, out=None, workspace: Optional[torch.Tensor] = None):
    """Keeps at most ``budget`` keys of every (sequence, head): the ``recent``
    last ones by position and those of the largest accumulated weight
    (instagen_evict).  k_cache, v_cache [B, Hkv, cap, d], weights [B, Hkv, cap]
    fp32, pos [B, Hkv, cap] int32, lens [B] int32.  In place, or into ``out``:
    (k, v, weights, pos, lens) with their own number of slots.  Returns the
    five evicted tensors."""
    dt = _dtype_of(k_cache, "k_cache")
    B, Hkv, cap, d = _cache_shape(k_cache, "k_cache", dt)
    _need(v_cache, "v_cache", dt, k_cache.shape)
    _need(weights, "weights", torch.float32, (B, Hkv, cap))
    _need(pos, "pos", torch.int32, (B, Hkv, cap))
    _need(lens, "lens", torch.int32, (B,))
    if out is None:
        out, cap_out = (k_cache, v_cache, weights, pos, lens), cap
    else:
        ko, vo, wo, po, lo = out
        cap_out = _cache_shape(ko, "out[0]", dt)[2]
        _need(ko, "out[0]", dt, (B, Hkv, cap_out, d))
        _need(vo, "out[1]", dt, (B, Hkv, cap_out, d))
        _need(wo, "out[2]", torch.float32, (B, Hkv, cap_out))
        _need(po, "out[3]", torch.int32, (B, Hkv, cap_out))
        _need(lo, "out[4]", torch.int32, (B,))
    if not 1 <= budget <= cap_out:
        raise ValueError(f"budget must be within [1, {cap_out}], got {budget}")
    if recent < 0:
        raise ValueError(f"recent must be >= 0, got {recent}")
    _on_current(k_cache, v_cache, weights, pos, lens, *out)
    p = CacheParams(B, Hkv, Hkv, d, 0, cap, _DTYPES[dt], 1.0, Hkv * d, 0)
    L, ref = lib(), ctypes.byref(p)
    ws, nws = _work_area(workspace, L.instagen_evict_workspace_size(ref, budget), k_cache, "instagen_evict")
    _check(L.instagen_evict(_ptr(k_cache), _ptr(v_cache), _ptr(weights), _ptr(pos), _ptr(lens), ref, budget,
                            min(recent, 2 ** 31 - 1), _ptr(out[0]), _ptr(out[1]), _ptr(out[2]), _ptr(out[3]),
                            _ptr(out[4]), cap_out, _ptr(ws), nws, _stream()), "instagen_evict")
    return tuple(out)
