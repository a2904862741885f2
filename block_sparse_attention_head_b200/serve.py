"""Binding of the language-model entry points of ``libinstagen.so``:
``prompt_attention``, ``key_weights``, ``prefix_attention`` and ``evict``
(argument marshalling only; the contracts are in ``include/instagen.h``).

A call for a few short sequences runs for some microseconds on the GPU, so the
marshalling is kept short: every check is made once, a tensor that fails one is
handed to a slower function that says why, and the parameter blocks are packed
as the C structs lay them out (``PromptParams``, ``CacheParams``)."""
from __future__ import annotations

import struct
from typing import Optional

import torch

from . import InstaGenError, _check, _need, lib

_DTYPES = {torch.bfloat16: 0, torch.float16: 1}  # instagen_dtype
_F32, _I32, _U8 = torch.float32, torch.int32, torch.uint8
_prompt_block = struct.Struct("@8if4x8q").pack  # instagen_prompt_params
_cache_block = struct.Struct("@7if2q").pack     # instagen_cache_params


def _device(t, name: str) -> int:
    """The current device, given that t is a CUDA tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise InstaGenError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    return torch._C._cuda_getDevice()


def _stream(dev: int) -> int:
    return torch._C._cuda_getCurrentRawStream(dev)


def _wrong_device(t, dev):
    raise InstaGenError(f"tensors must be on the current device cuda:{dev}, got {t.device}")


def _dtype_of(t, name: str):
    if not isinstance(t, torch.Tensor) or t.dtype not in _DTYPES:
        raise TypeError(f"{name} must be a bfloat16 or float16 torch.Tensor")
    return t.dtype


def _flat(t, name: str, dtype, shape, dev: int) -> int:
    """Address of a contiguous tensor of this type and shape on device dev."""
    if not (isinstance(t, torch.Tensor) and t.get_device() == dev and t.dtype is dtype and t.shape == shape
            and t.is_contiguous()):
        _need(t, name, dtype, shape)
        _wrong_device(t, dev)
    return t.data_ptr()


def _rows(t, name: str, dtype, shape, dev: int):
    """Address and strides of a 3-D tensor of rows: last dimension contiguous,
    the others strided in whole 16-byte steps without overlap."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != dev:
        if not t.is_cuda:
            raise InstaGenError(f"{name} must be a CUDA tensor (the library has no CPU path)")
        _wrong_device(t, dev)
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    n0, n1, d = shape
    s0, s1, s2 = t.stride()
    if s2 != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    if (n0 > 1 and (s0 < d or s0 % 8)) or (n1 > 1 and (s1 < d or s1 % 8)):
        raise ValueError(f"{name}: strides must be multiples of 8 elements and at least a row, got {t.stride()}")
    return t.data_ptr(), s0, s1


def _cache_shape(t, name: str, dtype):
    if not isinstance(t, torch.Tensor) or t.dim() != 4:
        _need(t, name, dtype)
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected [B, Hkv, slots, d]")
    return t.shape


def _heads(Hq: int, Hkv: int):
    if Hkv < 1 or Hq < 1 or Hq % Hkv:
        raise ValueError(f"{Hq} query heads cannot share {Hkv} key/value heads")


def _work_area(workspace: Optional[torch.Tensor], need: int, like: torch.Tensor, dev: int, what: str):
    if need == 0:
        raise InstaGenError(f"invalid or unsupported parameters for {what}")
    if workspace is None:
        if need == 256:  # the call needs no scratch
            return None, None, 0
        workspace = like.new_empty((need,), dtype=_U8)
        return workspace, workspace.data_ptr(), need
    have = workspace.numel() * workspace.element_size()
    if have < need:
        raise InstaGenError(f"workspace too small: {have} < {need}")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    if workspace.get_device() != dev:
        _wrong_device(workspace, dev)
    return workspace, workspace.data_ptr(), have


def _prompt_shapes(q, k, cu_q, cu_k, dev: int):
    dt = _dtype_of(q, "q")
    if not isinstance(k, torch.Tensor):
        raise TypeError("k must be a torch.Tensor")
    qs, ks = q.shape, k.shape
    if len(qs) != 3 or len(ks) != 3 or ks[2] != qs[2]:
        raise ValueError(f"q {tuple(qs)} and k {tuple(ks)} must be [Tq, Hq, d] and [Tk, Hkv, d]")
    _heads(qs[1], ks[1])
    if not isinstance(cu_q, torch.Tensor) or cu_q.dim() != 1 or cu_q.shape[0] < 2:
        _need(cu_q, "cu_q", _I32)
        raise ValueError("cu_q must hold the starts of the sequences and the end of the last one")
    ends = cu_q.shape
    return dt, qs, ks, ends[0] - 1, _flat(cu_q, "cu_q", _I32, ends, dev), _flat(cu_k, "cu_k", _I32, ends, dev)


def prompt_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_q: torch.Tensor, cu_k: torch.Tensor, *,
                     causal: bool = True, softmax_scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                     lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """Attention over packed prompts (instagen_prompt_attention): q [Tq, Hq, d],
    k and v [Tk, Hkv, d] bf16 or fp16 (views with 16-byte strides are read in
    place), cu_q and cu_k int32 [sequences + 1].  Query i of a sequence sees its
    keys j <= i + n_k - n_q (causal) or all of them.  Returns (O [Tq, Hq, d], lse
    [Hq, Tq] fp32); a row without keys is 0 with lse -inf.  Rows that belong to
    no sequence are not written (undefined unless ``out`` and ``lse`` are given)."""
    dev = _device(q, "q")
    dt, qs, ks, nseq, cq, ck = _prompt_shapes(q, k, cu_q, cu_k, dev)
    (Tq, Hq, d), (Tk, Hkv, _) = qs, ks
    qp, q0, q1 = _rows(q, "q", dt, qs, dev)
    kp, k0, k1 = _rows(k, "k", dt, ks, dev)
    vp, v0, v1 = _rows(v, "v", dt, ks, dev)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
        op, o0, o1 = out.data_ptr(), Hq * d, d
    else:
        op, o0, o1 = _rows(out, "out", dt, qs, dev)
    if lse is None:
        lse = q.new_empty((Hq, Tq), dtype=_F32)
        lp = lse.data_ptr()
    else:
        lp = _flat(lse, "lse", _F32, (Hq, Tq), dev)
    L = lib()
    p = _prompt_block(nseq, Hq, Hkv, d, Tq, Tk, _DTYPES[dt], 1 if causal else 0,
                      d ** -0.5 if softmax_scale is None else softmax_scale, q0, q1, k0, k1, v0, v1, o0, o1)
    workspace, ws, nws = _work_area(workspace, L.instagen_prompt_attention_workspace_size(p), q, dev,
                                    "instagen_prompt_attention")
    rc = L.instagen_prompt_attention(qp, kp, vp, cq, ck, p, op, lp, ws, nws, _stream(dev))
    if rc:
        _check(rc, "instagen_prompt_attention")
    return out, lse


def key_weights(q: torch.Tensor, k: torch.Tensor, lse: torch.Tensor, cu_q: torch.Tensor, cu_k: torch.Tensor,
                weights: torch.Tensor, *, causal: bool = True, softmax_scale: Optional[float] = None,
                workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Adds to weights [Hkv, Tk] fp32 what every key gets of the queries'
    attention, summed over the queries that see it and the heads that share it
    (instagen_key_weights).  lse [Hq, Tq]: as ``prompt_attention`` returned it
    for these queries.  Returns weights."""
    dev = _device(q, "q")
    dt, qs, ks, nseq, cq, ck = _prompt_shapes(q, k, cu_q, cu_k, dev)
    (Tq, Hq, d), (Tk, Hkv, _) = qs, ks
    qp, q0, q1 = _rows(q, "q", dt, qs, dev)
    kp, k0, k1 = _rows(k, "k", dt, ks, dev)
    lp = _flat(lse, "lse", _F32, (Hq, Tq), dev)
    wp = _flat(weights, "weights", _F32, (Hkv, Tk), dev)
    L = lib()
    p = _prompt_block(nseq, Hq, Hkv, d, Tq, Tk, _DTYPES[dt], 1 if causal else 0,
                      d ** -0.5 if softmax_scale is None else softmax_scale, q0, q1, k0, k1, k0, k1, q0, q1)
    workspace, ws, nws = _work_area(workspace, L.instagen_key_weights_workspace_size(p), q, dev,
                                    "instagen_key_weights")
    rc = L.instagen_key_weights(qp, kp, lp, cq, ck, p, wp, ws, nws, _stream(dev))
    if rc:
        _check(rc, "instagen_key_weights")
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
    dev = _device(q, "q")
    dt = _dtype_of(q, "q")
    cs = _cache_shape(k_cache, "k_cache", dt)
    B, Hkv, cap, d = cs
    kc, vc = _flat(k_cache, "k_cache", dt, cs, dev), _flat(v_cache, "v_cache", dt, cs, dev)
    qs = q.shape
    if len(qs) != 3 or qs[0] != B or qs[2] != d:
        raise ValueError(f"q has shape {tuple(qs)}, expected ({B}, Hq, {d})")
    Hq = qs[1]
    _heads(Hq, Hkv)
    qp, q0, q1 = _rows(q, "q", dt, qs, dev)
    if Hq > 1 and q1 != d:
        raise ValueError("q: the heads of a token must be contiguous")
    if (k_prefix is None) != (v_prefix is None):
        raise ValueError("k_prefix and v_prefix come together")
    P, kp, vp, ph = 0, None, None, 0
    if k_prefix is not None:
        if not isinstance(k_prefix, torch.Tensor) or k_prefix.dim() != 3:
            raise ValueError("k_prefix must be a tensor [Hkv, P, d]")
        P = k_prefix.shape[1]
        kp, ph, k1 = _rows(k_prefix, "k_prefix", dt, (Hkv, P, d), dev)
        vp, vh, v1 = _rows(v_prefix, "v_prefix", dt, (Hkv, P, d), dev)
        if P > 1 and (k1 != d or v1 != d):
            raise ValueError("k_prefix, v_prefix: the rows of a head must be contiguous")
        if Hkv > 1 and P > 0 and vh != ph:
            raise ValueError("k_prefix and v_prefix must have the same strides")
    np = _flat(lens, "lens", _I32, (B,), dev)
    wp = None if weights is None else _flat(weights, "weights", _F32, (B, Hkv, cap), dev)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
        op = out.data_ptr()
    else:
        op = _flat(out, "out", dt, qs, dev)
    if lse is None:
        lse = q.new_empty((B, Hq), dtype=_F32)
        lp = lse.data_ptr()
    else:
        lp = _flat(lse, "lse", _F32, (B, Hq), dev)
    L = lib()
    p = _cache_block(B, Hq, Hkv, d, P, cap, _DTYPES[dt], d ** -0.5 if softmax_scale is None else softmax_scale, q0, ph)
    workspace, ws, nws = _work_area(workspace, L.instagen_prefix_attention_workspace_size(p, wp is not None), q, dev,
                                    "instagen_prefix_attention")
    rc = L.instagen_prefix_attention(qp, kp, vp, kc, vc, np, p, op, lp, wp, ws, nws, _stream(dev))
    if rc:
        _check(rc, "instagen_prefix_attention")
    return out, lse


def evict(k_cache: torch.Tensor, v_cache: torch.Tensor, weights: torch.Tensor, pos: torch.Tensor, lens: torch.Tensor,
          budget: int, recent: int, *, out=None, workspace: Optional[torch.Tensor] = None):
    """Keeps at most ``budget`` keys of every (sequence, head): the ``recent``
    last ones by position and those of the largest accumulated weight
    (instagen_evict).  k_cache, v_cache [B, Hkv, cap, d], weights [B, Hkv, cap]
    fp32, pos [B, Hkv, cap] int32, lens [B] int32.  In place, or into ``out``:
    (k, v, weights, pos, lens) with their own number of slots.  Returns the
    five evicted tensors."""
    dev = _device(k_cache, "k_cache")
    dt = _dtype_of(k_cache, "k_cache")
    cs = _cache_shape(k_cache, "k_cache", dt)
    B, Hkv, cap, d = cs
    ins = (_flat(k_cache, "k_cache", dt, cs, dev), _flat(v_cache, "v_cache", dt, cs, dev),
           _flat(weights, "weights", _F32, (B, Hkv, cap), dev), _flat(pos, "pos", _I32, (B, Hkv, cap), dev),
           _flat(lens, "lens", _I32, (B,), dev))
    if out is None:
        out, outs, cap_out = (k_cache, v_cache, weights, pos, lens), ins, cap
    else:
        ko, vo, wo, po, lo = out
        os = _cache_shape(ko, "out[0]", dt)
        cap_out = os[2]
        os = (B, Hkv, cap_out, d)
        outs = (_flat(ko, "out[0]", dt, os, dev), _flat(vo, "out[1]", dt, os, dev),
                _flat(wo, "out[2]", _F32, (B, Hkv, cap_out), dev), _flat(po, "out[3]", _I32, (B, Hkv, cap_out), dev),
                _flat(lo, "out[4]", _I32, (B,), dev))
    if not 1 <= budget <= cap_out:
        raise ValueError(f"budget must be within [1, {cap_out}], got {budget}")
    if recent < 0:
        raise ValueError(f"recent must be >= 0, got {recent}")
    L = lib()
    p = _cache_block(B, Hkv, Hkv, d, 0, cap, _DTYPES[dt], 1.0, Hkv * d, 0)
    workspace, ws, nws = _work_area(workspace, L.instagen_evict_workspace_size(p, budget), k_cache, dev,
                                    "instagen_evict")
    rc = L.instagen_evict(*ins, p, budget, min(recent, 2 ** 31 - 1), *outs, cap_out, ws, nws, _stream(dev))
    if rc:
        _check(rc, "instagen_evict")
    return tuple(out)
