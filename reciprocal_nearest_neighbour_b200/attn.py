"""Binding of the attention entry points: argument checks and marshalling.

``kv_append`` puts new tokens' keys and values into a paged cache (rotating
keys and queries by their positions), ``attn_prompt`` attends within packed
sequences, ``attn_decode`` attends from one new token per sequence over the
cache.  Tensors are fp16 or bf16 CUDA tensors whose last dimension (the
channels of a head) is contiguous; the other dimensions may have any strides
that are multiples of 8 elements, so slices of a fused projection's output
pass as they are.  Calls run on the current stream of the tensors' device.
"""
from __future__ import annotations

import math
from typing import Optional

import torch

from . import _lib

_DT = {torch.float16: _lib.RNN_F16, torch.bfloat16: _lib.RNN_BF16}


def _check(t, name: str, ndim: int, dtype, device=None) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got shape {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _value_dtype(t, name: str):
    if not isinstance(t, torch.Tensor) or t.dtype not in _DT:
        raise TypeError(f"{name} must be float16 or bfloat16, got "
                        f"{getattr(t, 'dtype', type(t).__name__)}")
    return t.dtype


def _strides(t: torch.Tensor, name: str):
    """Element strides of the leading dimensions, the channels being contiguous."""
    d = t.shape[-1]
    if t.stride(-1) != 1 and d > 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    out = []
    for size, stride in zip(t.shape[:-1], t.stride()[:-1]):
        if size <= 1:
            stride = d
        elif stride < d or stride % 8:
            raise ValueError(f"strides of {name} must be multiples of 8 elements and at least "
                             f"{d}, got {tuple(t.stride())}")
        out.append(stride)
    if t.data_ptr() % 16:
        raise ValueError(f"{name} must start on a 16-byte boundary")
    return out


def _rows(t: Optional[torch.Tensor], name: str) -> _lib.Rows:
    if t is None:
        return _lib.Rows(None, 0, 0)
    token, head = _strides(t, name)
    return _lib.Rows(t.data_ptr(), token, head)


def _pages(t: torch.Tensor, name: str) -> _lib.Pages:
    return _lib.Pages(t.data_ptr(), *_strides(t, name))


def _ints(t, name: str, device, size: int) -> None:
    _check(t, name, 1, torch.int32, device)
    if t.shape[0] != size:
        raise ValueError(f"{name} must have {size} values, got {t.shape[0]}")
    if size > 1 and t.stride(0) != 1:
        raise ValueError(f"{name} must be contiguous")


def _cu(t, name: str, device) -> int:
    _check(t, name, 1, torch.int32, device)
    if t.shape[0] < 1:
        raise ValueError(f"{name} must have one value more than there are sequences")
    _ints(t, name, device, t.shape[0])
    return t.shape[0] - 1


def _table(t, device, B: int):
    _check(t, "page_table", 2, torch.int32, device)
    if t.shape[0] != B or t.shape[1] < 1:
        raise ValueError(f"page_table must have shape [{B}, pages >= 1], got {tuple(t.shape)}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("rows of page_table must be contiguous")
    return t.stride(0) if B > 1 else t.shape[1]


def _cache(k_cache, v_cache, kind, device, heads: int, d: int) -> None:
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _check(t, name, 4, kind, device)
        if t.shape[2:] != (heads, d) or t.shape[0] < 1 or t.shape[1] < 1:
            raise ValueError(f"{name} must have shape [pages, page_size, {heads}, {d}], got "
                             f"{tuple(t.shape)}")
    if k_cache.shape != v_cache.shape:
        raise ValueError("k_cache and v_cache must have the same shape")


def _heads(hq: int, hkv: int, d: int, d_max: int) -> None:
    if hkv < 1 or hq < 1 or hq % hkv:
        raise ValueError(f"query heads ({hq}) must be a multiple of key heads ({hkv})")
    if d < 8 or d % 8 or d > d_max:
        raise ValueError(f"channels per head must be a multiple of 8 up to {d_max}, got {d}")
    if hq > _lib.RNN_ATTN_MAX_HEADS:
        raise ValueError(f"at most {_lib.RNN_ATTN_MAX_HEADS} heads, got {hq}")


def _scale(scale: Optional[float], d: int) -> float:
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    if not (scale > 0.0 and scale < 3e38):
        raise ValueError(f"scale must be positive and finite, got {scale}")
    return scale


def _like(out, want: torch.Size, kind, device, name: str) -> torch.Tensor:
    if out is None:
        return torch.empty(want, dtype=kind, device=device)
    _check(out, name, len(want), kind, device)
    if out.shape != want:
        raise ValueError(f"{name} must have shape {tuple(want)}, got {tuple(out.shape)}")
    return out


def _scratch(workspace, need: int, device) -> torch.Tensor:
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    if not isinstance(workspace, torch.Tensor) or workspace.device != device or \
            workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {device}")
    return workspace


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def kv_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
              page_table: torch.Tensor, start: torch.Tensor, cu: torch.Tensor, *,
              q: Optional[torch.Tensor] = None, inv_freq: Optional[torch.Tensor] = None,
              positions: Optional[torch.Tensor] = None, paired: bool = False,
              with_k: bool = False, q_out: Optional[torch.Tensor] = None,
              k_out: Optional[torch.Tensor] = None):
    """Append packed new tokens ``k, v [T, Hkv, d]`` to the caches ``[pages, page_size, Hkv, d]``.

    Sequence ``b`` has the tokens ``cu[b]:cu[b+1]`` and ``start[b]`` tokens in
    the cache already; ``page_table [B, n]`` names its pages (all int32).
    With ``inv_freq`` (float64 ``[pairs]``) the keys, and the queries ``q [T,
    Hq, d]`` if given, are turned by ``position * inv_freq``: the position is
    the token's number in its sequence, or ``positions`` (int32 ``[T]``, or
    ``[T, 2]`` for the row and column of a patch, each turning half of the
    rotated channels).  ``paired`` pairs channels ``2i, 2i+1`` instead of
    ``i, pairs+i``.

    Returns ``(q_out, k_out)``: the rotated queries (``None`` without ``q``)
    and, ``with_k`` or into a given ``k_out``, the rotated keys packed like
    ``k`` (``None`` otherwise).  ``q_out=q`` and ``k_out=k`` rotate in place.
    Rows outside the sequences are not written; a token whose page does not
    exist is not stored.
    """
    kind = _value_dtype(k, "k")
    _check(k, "k", 3, kind)
    dev = k.device
    T, hkv, d = k.shape
    _check(v, "v", 3, kind, dev)
    if v.shape != k.shape:
        raise ValueError(f"v must have the shape of k, got {tuple(v.shape)}")
    hq = 0
    if q is not None:
        _check(q, "q", 3, kind, dev)
        hq = q.shape[1]
        if q.shape[0] != T or q.shape[2] != d or hq < 1:
            raise ValueError(f"q must have shape [{T}, heads, {d}], got {tuple(q.shape)}")
        if inv_freq is None:
            raise ValueError("q is only rotated: it needs inv_freq")
    elif q_out is not None:
        raise ValueError("q_out needs q")
    if hkv < 1 or d < 8 or d % 8 or d > 256:
        raise ValueError(f"channels per head must be a multiple of 8 up to 256, got {d}")
    if max(hq, hkv) > _lib.RNN_ATTN_MAX_HEADS:
        raise ValueError(f"at most {_lib.RNN_ATTN_MAX_HEADS} heads")
    _cache(k_cache, v_cache, kind, dev, hkv, d)
    B = _cu(cu, "cu", dev)
    _ints(start, "start", dev, B)
    table_stride = _table(page_table, dev, B)
    pairs = axes = pos_stride = 0
    if inv_freq is not None:
        _check(inv_freq, "inv_freq", 1, torch.float64, dev)
        pairs, axes = inv_freq.shape[0], 1
        if pairs < 1 or (pairs > 1 and inv_freq.stride(0) != 1):
            raise ValueError("inv_freq must be contiguous and not empty")
    if positions is not None:
        if inv_freq is None:
            raise ValueError("positions need inv_freq")
        if not isinstance(positions, torch.Tensor) or positions.dim() not in (1, 2):
            raise ValueError("positions must be a [T] or [T, 2] tensor")
        _check(positions, "positions", positions.dim(), torch.int32, dev)
        axes = positions.shape[1] if positions.dim() == 2 else 1
        if positions.shape[0] != T or axes not in (1, 2):
            raise ValueError(f"positions must have shape [{T}] or [{T}, 2], got "
                             f"{tuple(positions.shape)}")
        if positions.dim() == 2 and axes > 1 and positions.stride(1) != 1:
            raise ValueError("rows of positions must be contiguous")
        pos_stride = positions.stride(0) if T > 1 else axes
        if pos_stride < axes:
            raise ValueError("rows of positions must not overlap")
    if 2 * pairs * axes > d:
        raise ValueError(f"{2 * pairs * axes} rotated channels do not fit into {d}")
    if q is not None:
        q_out = _like(q_out, q.shape, kind, dev, "q_out")
    if with_k or k_out is not None:
        k_out = _like(k_out, k.shape, kind, dev, "k_out")
    lib = _lib.load()
    with torch.cuda.device(dev):
        _lib.check(lib.rnn_kv_append(
            _rows(q, "q"), _rows(k, "k"), _rows(v, "v"), T, hq, hkv, d, _DT[kind],
            _pages(k_cache, "k_cache"), _pages(v_cache, "v_cache"), k_cache.shape[0],
            k_cache.shape[1], page_table.data_ptr(), table_stride, page_table.shape[1],
            start.data_ptr(), cu.data_ptr(), B,
            None if positions is None else positions.data_ptr(), pos_stride,
            None if inv_freq is None else inv_freq.data_ptr(), pairs, axes, int(paired),
            _rows(q_out, "q_out"), _rows(k_out, "k_out"), _stream(dev)), "rnn_kv_append")
    return q_out, k_out


def attn_prompt(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_q: torch.Tensor,
                cu_k: Optional[torch.Tensor] = None, *, causal: bool = True,
                scale: Optional[float] = None, with_lse: bool = False,
                out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """Attention of packed sequences: ``q [Tq, Hq, d]`` over ``k, v [Tk, Hkv, d]``.

    Sequence ``b`` has the queries ``cu_q[b]:cu_q[b+1]`` and the keys
    ``cu_k[b]:cu_k[b+1]`` (int32 on the device; ``cu_k`` defaults to
    ``cu_q``).  ``causal``: query ``i`` of ``nq`` sees the keys up to ``i + nk
    - nq``; else all keys of its sequence.  ``scale`` defaults to ``1/sqrt(d)``.
    Query head ``h`` reads key head ``h // (Hq // Hkv)``.

    Returns ``out [Tq, Hq, d]``, or ``(out, lse)`` with ``lse [Tq, Hq]`` float32
    the log-sum-exp of the scaled scores.  A row that sees no key is 0 with
    ``lse`` -inf; rows outside the sequences are not written.
    """
    kind = _value_dtype(q, "q")
    _check(q, "q", 3, kind)
    dev = q.device
    _check(k, "k", 3, kind, dev)
    _check(v, "v", 3, kind, dev)
    Tq, hq, d = q.shape
    Tk, hkv = k.shape[:2]
    if k.shape != v.shape or k.shape[2] != d:
        raise ValueError(f"k and v must have shape [tokens, heads, {d}], got {tuple(k.shape)} "
                         f"and {tuple(v.shape)}")
    _heads(hq, hkv, d, _lib.RNN_ATTN_MAX_DIM)
    B = _cu(cu_q, "cu_q", dev)
    if cu_k is None:
        cu_k = cu_q
    _ints(cu_k, "cu_k", dev, B + 1)
    scale = _scale(scale, d)
    out = _like(out, q.shape, kind, dev, "out")
    lse = torch.empty((Tq, hq), dtype=torch.float32, device=dev) if with_lse else None
    lib = _lib.load()
    ws = _scratch(workspace, lib.rnn_attn_prompt_workspace_size(), dev)
    with torch.cuda.device(dev):
        _lib.check(lib.rnn_attn_prompt(
            _rows(q, "q"), _rows(k, "k"), _rows(v, "v"), Tq, Tk, hq, hkv, d, _DT[kind],
            cu_q.data_ptr(), cu_k.data_ptr(), B, int(causal), scale, _rows(out, "out"),
            None if lse is None else lse.data_ptr(), ws.data_ptr(), ws.numel(), _stream(dev)),
            "rnn_attn_prompt")
    return (out, lse) if with_lse else out


def attn_decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                page_table: torch.Tensor, lens: torch.Tensor, *, scale: Optional[float] = None,
                with_lse: bool = False, out: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None):
    """Attention of one new token per sequence, ``q [B, Hq, d]``, over a paged cache.

    The caches are ``[pages, page_size, Hkv, d]``; sequence ``b`` has ``lens[b]``
    tokens (the new one included) on the pages ``page_table[b]`` (int32).
    ``scale``, heads and results as in ``attn_prompt``: ``out [B, Hq, d]``, or
    ``(out, lse [B, Hq])``.
    """
    kind = _value_dtype(q, "q")
    _check(q, "q", 3, kind)
    dev = q.device
    B, hq, d = q.shape
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache must be a [pages, page_size, heads, d] tensor")
    hkv = k_cache.shape[2]
    _heads(hq, hkv, d, _lib.RNN_ATTN_MAX_DIM)
    _cache(k_cache, v_cache, kind, dev, hkv, d)
    _ints(lens, "lens", dev, B)
    table_stride = _table(page_table, dev, B)
    scale = _scale(scale, d)
    out = _like(out, q.shape, kind, dev, "out")
    lse = torch.empty((B, hq), dtype=torch.float32, device=dev) if with_lse else None
    lib = _lib.load()
    ws = _scratch(workspace, lib.rnn_attn_decode_workspace_size(B, hq, hkv, d), dev)
    with torch.cuda.device(dev):
        _lib.check(lib.rnn_attn_decode(
            _rows(q, "q"), _pages(k_cache, "k_cache"), _pages(v_cache, "v_cache"),
            k_cache.shape[0], k_cache.shape[1], page_table.data_ptr(), table_stride,
            page_table.shape[1], lens.data_ptr(), B, hq, hkv, d, _DT[kind], scale,
            _rows(out, "out"), None if lse is None else lse.data_ptr(), ws.data_ptr(),
            ws.numel(), _stream(dev)), "rnn_attn_decode")
    return (out, lse) if with_lse else out
