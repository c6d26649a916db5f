"""Binding of the attention entry points: argument checks and marshalling.

``kv_append`` puts new tokens' keys and values into a paged cache (rotating
keys and queries by their positions), ``attn_prompt`` attends within packed
sequences, ``attn_decode`` attends from one new token per sequence over the
cache.  Tensors are fp16 or bf16 CUDA tensors whose last dimension (the
channels of a head) is contiguous; the other dimensions may have any strides
that are multiples of 8 elements, so slices of a fused projection's output
pass as they are (no two rows of an output may overlap).  Calls run on the
current stream of the tensors' device, and their results carry no gradient.
"""
from __future__ import annotations

import functools
import math
import struct
from typing import Optional

import torch

from . import _lib

_DT = {torch.float16: _lib.RNN_F16, torch.bfloat16: _lib.RNN_BF16}

# The argument structures of the C entry points (KvAppendArgs, AttnPromptArgs and AttnDecodeArgs of
# _lib), packed in one step: a ctypes structure filled field by field takes microseconds.
_ROWS, _PAGES = "Qqq", "Qqqq"
_APPEND = struct.Struct("=" + 5 * _ROWS + 2 * _PAGES + "5Q4q10i")
_PROMPT = struct.Struct("=" + 4 * _ROWS + "4QQ2q6if4x")
_DECODE = struct.Struct("=" + 2 * _ROWS + 2 * _PAGES + "4QQ2q7if")


def _check(t, name: str, ndim: int, dtype, device=None) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got shape {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _all(kind, device, ndim: int, *named) -> None:
    """Each ``tensor, name`` has this type, device and number of dimensions (else the error)."""
    for t in named[::2]:
        if not (isinstance(t, torch.Tensor) and t.dtype is kind and t.device == device
                and t.dim() == ndim and t.is_cuda):
            for u, name in zip(named[::2], named[1::2]):
                _check(u, name, ndim, kind, device)


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


_NO_ROWS = (0, 0, 0)


def _rows(t: torch.Tensor, name: str, d: int):
    token, head, one = t.stride()
    at = t.data_ptr()
    if one != 1 or token < d or head < d or (token | head) & 7 or at & 15:
        token, head = _strides(t, name)     # a dimension of size 1, or an error
    return at, token, head


def _pages(t: torch.Tensor, name: str, d: int):
    page, token, head, one = t.stride()
    at = t.data_ptr()
    if one != 1 or page < d or token < d or head < d or (page | token | head) & 7 or at & 15:
        page, token, head = _strides(t, name)
    return at, page, token, head


def _ints(t, name: str, device, size: int) -> None:
    if _cu(t, name, device, 0) != size - 1:
        raise ValueError(f"{name} must have {size} values, got {t.shape[0]}")


def _cu(t, name: str, device, least: int = 1) -> int:
    if not (isinstance(t, torch.Tensor) and t.dtype is torch.int32 and t.device == device
            and t.dim() == 1 and t.is_cuda):
        _check(t, name, 1, torch.int32, device)
    n, = t.shape
    if n < least:
        raise ValueError(f"{name} must have one value more than there are sequences")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return n - 1


def _table(t, device, B: int):
    """Row stride and row length of the page table."""
    _check(t, "page_table", 2, torch.int32, device)
    rows, n = t.shape
    if rows != B or n < 1:
        raise ValueError(f"page_table must have shape [{B}, pages >= 1], got {tuple(t.shape)}")
    stride, one = t.stride()
    if n > 1 and one != 1:
        raise ValueError("rows of page_table must be contiguous")
    return (stride if B > 1 else n), n


def _cache(k_cache, v_cache, kind, device, heads: int, d: int):
    """Number of pages and page size."""
    _all(kind, device, 4, k_cache, "k_cache", v_cache, "v_cache")
    pages, size, h, dim = shape = k_cache.shape
    if h != heads or dim != d or pages < 1 or size < 1:
        raise ValueError(f"k_cache must have shape [pages, page_size, {heads}, {d}], got "
                         f"{tuple(shape)}")
    if shape != v_cache.shape:
        raise ValueError("k_cache and v_cache must have the same shape")
    return pages, size


def _heads(hq: int, hkv: int, d: int, d_max: int) -> None:
    if hkv < 1 or hq < 1 or hq % hkv:
        raise ValueError(f"query heads ({hq}) must be a multiple of key heads ({hkv})")
    if d < 8 or d % 8 or d > d_max:
        raise ValueError(f"channels per head must be a multiple of 8 up to {d_max}, got {d}")
    if hq > _lib.RNN_ATTN_MAX_HEADS:
        raise ValueError(f"at most {_lib.RNN_ATTN_MAX_HEADS} heads, got {hq}")


def _scale(scale: Optional[float], d: int) -> float:
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    if not 0.0 < scale < 2e38:
        raise ValueError(f"scale must be positive and below 2e38, got {scale}")
    return scale


def _packed(t: torch.Tensor) -> torch.Tensor:
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _given(out, want: torch.Size, kind, device, name: str) -> torch.Tensor:
    _check(out, name, len(want), kind, device)
    if out.shape != want:
        raise ValueError(f"{name} must have shape {tuple(want)}, got {tuple(out.shape)}")
    return out


def _given_scratch(workspace, device):
    """Address and size of the caller's workspace, or none."""
    if workspace is None:
        return 0, 0
    if not isinstance(workspace, torch.Tensor) or workspace.device != device or \
            workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {device}")
    return workspace.data_ptr(), workspace.numel()


@functools.lru_cache(maxsize=256)
def _decode_need(B: int, hq: int, hkv: int, d: int) -> int:
    return _lib.load().rnn_attn_decode_workspace_size(B, hq, hkv, d)


def _call(fn, name: str, t: torch.Tensor, args: bytes) -> None:
    """``fn(args, stream)`` with the device of `t` current, on its current stream."""
    index = t.get_device()
    if index == torch._C._cuda_getDevice():
        code = fn(args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            code = fn(args, torch._C._cuda_getCurrentRawStream(index))
    if code:
        _lib.check(code, name)


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
    ``k`` (``None`` otherwise).  ``q_out=q`` and ``k_out=k`` rotate in place;
    otherwise outputs lie apart from the inputs.
    Rows outside the sequences are not written; a token whose page does not
    exist is not stored.
    """
    kind = _value_dtype(k, "k")
    dev = k.device
    _all(kind, dev, 3, k, "k", v, "v")
    T, hkv, d = shape = k.shape
    if v.shape != shape:
        raise ValueError(f"v must have the shape of k, got {tuple(v.shape)}")
    hq = 0
    if q is not None:
        _all(kind, dev, 3, q, "q")
        tq, hq, dq = q.shape
        if tq != T or dq != d or hq < 1:
            raise ValueError(f"q must have shape [{T}, heads, {d}], got {tuple(q.shape)}")
        if inv_freq is None:
            raise ValueError("q is only rotated: it needs inv_freq")
    elif q_out is not None:
        raise ValueError("q_out needs q")
    if hkv < 1:
        raise ValueError("k and v have no heads")
    if d < 8 or d % 8 or d > 256:
        raise ValueError(f"channels per head must be a multiple of 8 up to 256, got {d}")
    if max(hq, hkv) > _lib.RNN_ATTN_MAX_HEADS:
        raise ValueError(f"at most {_lib.RNN_ATTN_MAX_HEADS} heads")
    num_pages, size = _cache(k_cache, v_cache, kind, dev, hkv, d)
    B = _cu(cu, "cu", dev)
    _ints(start, "start", dev, B)
    table_stride, max_pages = _table(page_table, dev, B)
    pairs = axes = pos_stride = 0
    if inv_freq is not None:
        _all(torch.float64, dev, 1, inv_freq, "inv_freq")
        pairs, axes = inv_freq.shape[0], 1
        if pairs < 1 or not inv_freq.is_contiguous():
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
        q_out = _packed(q) if q_out is None else _given(q_out, q.shape, kind, dev, "q_out")
    if k_out is not None:
        _given(k_out, k.shape, kind, dev, "k_out")
    elif with_k:
        k_out = _packed(k)
    _call(_lib.load().rnn_kv_append, "rnn_kv_append", k, _APPEND.pack(
        *(_NO_ROWS if q is None else _rows(q, "q", d)), *_rows(k, "k", d), *_rows(v, "v", d),
        *(_NO_ROWS if q is None else _rows(q_out, "q_out", d)),
        *(_NO_ROWS if k_out is None else _rows(k_out, "k_out", d)),
        *_pages(k_cache, "k_cache", d), *_pages(v_cache, "v_cache", d), page_table.data_ptr(),
        start.data_ptr(), cu.data_ptr(), 0 if positions is None else positions.data_ptr(),
        0 if inv_freq is None else inv_freq.data_ptr(), T, num_pages, table_stride, pos_stride,
        hq, hkv, d, _DT[kind], size, max_pages, B, pairs, axes, bool(paired)))
    return q_out, k_out


def attn_prompt(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_q: torch.Tensor,
                cu_k: Optional[torch.Tensor] = None, *, causal: bool = True,
                scale: Optional[float] = None, with_lse: bool = False,
                out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """Attention of packed sequences: ``q [Tq, Hq, d]`` over ``k, v [Tk, Hkv, d]``, ``d <= 128``.

    Sequence ``b`` has the queries ``cu_q[b]:cu_q[b+1]`` and the keys
    ``cu_k[b]:cu_k[b+1]`` (int32 on the device; ``cu_k`` defaults to
    ``cu_q``).  ``causal``: query ``i`` of ``nq`` sees the keys up to ``i + nk
    - nq``; else all keys of its sequence.  ``scale`` defaults to ``1/sqrt(d)``.
    Query head ``h`` reads key head ``h // (Hq // Hkv)``.

    Returns ``out [Tq, Hq, d]`` (a given one lies apart from the inputs), or
    ``(out, lse)`` with ``lse [Tq, Hq]`` float32 the log-sum-exp of the scaled
    scores.  A row that sees no key is 0 with ``lse`` -inf, one that sees a score
    that is not a number is NaN; a value that is not finite may reach earlier
    rows of its sequence too.  Rows outside the sequences are not written.
    Should a wait of the kernel run out, the rows not computed are NaN; with a
    ``workspace`` (uint8, 256 bytes) ``workspace_status`` tells.
    """
    kind = _value_dtype(q, "q")
    dev = q.device
    _all(kind, dev, 3, q, "q", k, "k", v, "v")
    Tq, hq, d = q.shape
    Tk, hkv, dk = k.shape
    if dk != d or k.shape != v.shape:
        raise ValueError(f"k and v must have shape [tokens, heads, {d}], got {tuple(k.shape)} "
                         f"and {tuple(v.shape)}")
    _heads(hq, hkv, d, _lib.RNN_ATTN_MAX_DIM)
    B = _cu(cu_q, "cu_q", dev)
    if cu_k is None:
        cu_k = cu_q
    else:
        _ints(cu_k, "cu_k", dev, B + 1)
    scale = _scale(scale, d)
    out = _packed(q) if out is None else _given(out, q.shape, kind, dev, "out")
    lse = torch.empty((Tq, hq), dtype=torch.float32, device=dev) if with_lse else None
    ws, ws_bytes = _given_scratch(workspace, dev)
    _call(_lib.load().rnn_attn_prompt, "rnn_attn_prompt", q, _PROMPT.pack(
        *_rows(q, "q", d), *_rows(k, "k", d), *_rows(v, "v", d), *_rows(out, "out", d),
        cu_q.data_ptr(), cu_k.data_ptr(), 0 if lse is None else lse.data_ptr(), ws, ws_bytes, Tq,
        Tk, hq, hkv, d, _DT[kind], B, bool(causal), scale))
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
    dev = q.device
    _all(kind, dev, 3, q, "q")
    B, hq, d = q.shape
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache must be a [pages, page_size, heads, d] tensor")
    hkv = k_cache.shape[2]
    _heads(hq, hkv, d, _lib.RNN_ATTN_MAX_DIM)
    num_pages, size = _cache(k_cache, v_cache, kind, dev, hkv, d)
    _ints(lens, "lens", dev, B)
    table_stride, max_pages = _table(page_table, dev, B)
    scale = _scale(scale, d)
    out = _packed(q) if out is None else _given(out, q.shape, kind, dev, "out")
    lse = torch.empty((B, hq), dtype=torch.float32, device=dev) if with_lse else None
    if workspace is None:
        workspace = torch.empty(_decode_need(B, hq, hkv, d), dtype=torch.uint8, device=dev)
    ws, ws_bytes = _given_scratch(workspace, dev)
    _call(_lib.load().rnn_attn_decode, "rnn_attn_decode", q, _DECODE.pack(
        *_rows(q, "q", d), *_rows(out, "out", d), *_pages(k_cache, "k_cache", d),
        *_pages(v_cache, "v_cache", d), page_table.data_ptr(), lens.data_ptr(),
        0 if lse is None else lse.data_ptr(), ws, ws_bytes, num_pages, table_stride, size,
        max_pages, B, hq, hkv, d, _DT[kind], scale))
    return (out, lse) if with_lse else out
