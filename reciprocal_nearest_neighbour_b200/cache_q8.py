"""Binding of the cache in 8-bit codes: argument checks and marshalling.

``kv_append_q8`` is ``kv_append`` into a cache of codes, ``kv_read_q8`` gives
cached tokens back as packed 16-bit rows (for ``attn_prompt``), and
``attn_decode_q8`` is ``attn_decode`` over that cache.

The cache of a layer is three tensors: ``k_cache`` and ``v_cache [pages,
page_size, Hkv, d]`` of ``torch.float8_e4m3fn`` or ``torch.int8`` (whose
strides may be any multiples of 8), and ``scales [pages, Hkv, page_size, 2]``
float32, the key's and the value's scale of each token and head.  A row stands
for ``code * scale`` with ``scale = max(max|x| / top, 2**-126)``, ``top`` 448
(e4m3) or 127 (int8), and codes rounded to nearest.  Of values of one size
int8 keeps 1/254 of the row's largest, e4m3 1/16 of each value.
"""
from __future__ import annotations

import functools
import struct
from typing import Optional

import torch

from . import _lib
from .attn import (_DT, _NO_ROWS, _PAGES, _ROWS, _all, _call, _check, _cu, _given, _given_scratch,
                   _heads, _ints, _new_rows, _packed, _pages, _rotated, _rows, _scale, _strides,
                   _table, _turns, _value_dtype)

_CODES = {torch.float8_e4m3fn: _lib.RNN_CODES_E4M3, torch.int8: _lib.RNN_CODES_INT8}

# The argument structures of the C entry points, packed in one step.
_SCALES = "Qqq"
_APPEND = struct.Struct("=" + 5 * _ROWS + 2 * _PAGES + _SCALES + "5Q4q11i4x")
_READ = struct.Struct("=" + 2 * _ROWS + 2 * _PAGES + _SCALES + "3Q3q7i4x")
_DECODE = struct.Struct("=" + 2 * _ROWS + 2 * _PAGES + _SCALES + "4QQ2q8if4x")


def _coded(k_cache, v_cache, scales, device, heads: Optional[int], d: int):
    """Codes, heads, number of pages, page size, and the scales' address and strides."""
    if not isinstance(k_cache, torch.Tensor) or k_cache.dtype not in _CODES:
        raise TypeError("k_cache must be float8_e4m3fn or int8, got "
                        f"{getattr(k_cache, 'dtype', type(k_cache).__name__)}")
    _all(k_cache.dtype, device, 4, k_cache, "k_cache", v_cache, "v_cache")
    pages, size, h, dim = shape = k_cache.shape
    if (heads is not None and h != heads) or dim != d or pages < 1 or size < 1:
        raise ValueError(f"k_cache must have shape [pages, page_size, "
                         f"{'heads' if heads is None else heads}, {d}], got {tuple(shape)}")
    if shape != v_cache.shape:
        raise ValueError("k_cache and v_cache must have the same shape")
    _all(torch.float32, device, 4, scales, "scales")
    if scales.shape != (pages, h, size, 2):
        raise ValueError(f"scales must have shape {(pages, h, size, 2)}, got {tuple(scales.shape)}")
    page, head, row, one = scales.stride()
    if one != 1 or (row != 2 and size > 1):
        raise ValueError("a head's scales of a page must be contiguous")
    for n, s in ((pages, page), (h, head)):
        if n > 1 and (s < 2 * size or s % 2):
            raise ValueError(f"strides of scales must be even and at least {2 * size}, got "
                             f"{tuple(scales.stride())}")
    if scales.data_ptr() % 8:
        raise ValueError("scales must start on an 8-byte boundary")
    return _CODES[k_cache.dtype], h, pages, size, (scales.data_ptr(), page, head)


def kv_append_q8(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                 scales: torch.Tensor, page_table: torch.Tensor, start: torch.Tensor,
                 cu: torch.Tensor, *, q: Optional[torch.Tensor] = None,
                 inv_freq: Optional[torch.Tensor] = None,
                 positions: Optional[torch.Tensor] = None, paired: bool = False,
                 with_k: bool = False, q_out: Optional[torch.Tensor] = None,
                 k_out: Optional[torch.Tensor] = None):
    """``kv_append`` into a cache of codes and scales.

    The rotated keys are quantised from fp32, before any rounding to 16 bits;
    ``k_out`` has them in 16 bits, not as the cache holds them.  A row with a
    channel that is not finite reads back as NaN.  Outputs given in place of
    ``q`` and ``k`` have their strides.  All else is as in ``kv_append``.
    """
    done = (_lib.fast or _lib.load_fast()).kv_append_q8(
        k, v, k_cache, v_cache, scales, page_table, start, cu, q, inv_freq, positions, paired,
        with_k, q_out, k_out)
    if done is not None:
        return _lib.served(done, "rnn_kv_append_q8")
    kind, dev, T, hq, hkv, d = _new_rows(k, v, q, q_out, inv_freq)
    codes, _, num_pages, size, scale_at = _coded(k_cache, v_cache, scales, dev, hkv, d)
    B = _cu(cu, "cu", dev)
    _ints(start, "start", dev, B)
    table_stride, max_pages = _table(page_table, dev, B)
    pairs, axes, pos_stride = _turns(inv_freq, positions, T, d, dev)
    q_out, k_out = _rotated(q, k, q_out, k_out, with_k)
    _call(_lib.load().rnn_kv_append_q8, "rnn_kv_append_q8", k, _APPEND.pack(
        *(_NO_ROWS if q is None else _rows(q, "q", d)), *_rows(k, "k", d), *_rows(v, "v", d),
        *(_NO_ROWS if q is None else _rows(q_out, "q_out", d)),
        *(_NO_ROWS if k_out is None else _rows(k_out, "k_out", d)),
        *_pages(k_cache, "k_cache", d), *_pages(v_cache, "v_cache", d), *scale_at,
        page_table.data_ptr(), start.data_ptr(), cu.data_ptr(),
        0 if positions is None else positions.data_ptr(),
        0 if inv_freq is None else inv_freq.data_ptr(), T, num_pages, table_stride, pos_stride,
        hq, hkv, d, _DT[kind], codes, size, max_pages, B, pairs, axes, bool(paired)))
    return q_out, k_out


def kv_read_q8(k_cache: torch.Tensor, v_cache: torch.Tensor, scales: torch.Tensor,
               page_table: torch.Tensor, cu: torch.Tensor, tokens: int,
               dtype: torch.dtype = torch.bfloat16, *, start: Optional[torch.Tensor] = None,
               k_out: Optional[torch.Tensor] = None, v_out: Optional[torch.Tensor] = None):
    """Cached tokens as packed rows ``k, v [tokens, Hkv, d]`` of ``dtype``.

    Sequence ``b`` gives the rows ``cu[b]:cu[b+1]``, its tokens number
    ``start[b]`` and on (int32, default 0), placed by ``page_table [B, n]`` as in
    ``kv_append``; a token whose page does not exist gives zeros.  ``tokens`` is
    the number of packed rows; rows outside the sequences are not written.
    """
    if dtype not in _DT:
        raise TypeError(f"dtype must be float16 or bfloat16, got {dtype}")
    done = (_lib.fast or _lib.load_fast()).kv_read_q8(
        k_cache, v_cache, scales, page_table, cu, tokens, dtype is torch.bfloat16, start, k_out, v_out)
    if done is not None:
        return _lib.served(done, "rnn_kv_read_q8")
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache must be a [pages, page_size, heads, d] tensor")
    dev, d, tokens = k_cache.device, k_cache.shape[3], int(tokens)
    codes, hkv, num_pages, size, scale_at = _coded(k_cache, v_cache, scales, dev, None, d)
    if tokens < 0:
        raise ValueError(f"tokens must not be negative, got {tokens}")
    if hkv < 1 or hkv > _lib.RNN_ATTN_MAX_HEADS:
        raise ValueError(f"1 to {_lib.RNN_ATTN_MAX_HEADS} heads, got {hkv}")
    if d < 8 or d % 8 or d > 256:
        raise ValueError(f"channels per head must be a multiple of 8 up to 256, got {d}")
    B = _cu(cu, "cu", dev)
    if start is not None:
        _ints(start, "start", dev, B)
    table_stride, max_pages = _table(page_table, dev, B)
    want = torch.Size((tokens, hkv, d))
    outs = [torch.empty(want, dtype=dtype, device=dev) if out is None else
            _given(out, want, dtype, dev, name) for out, name in ((k_out, "k_out"), (v_out, "v_out"))]
    _call(_lib.load().rnn_kv_read_q8, "rnn_kv_read_q8", k_cache, _READ.pack(
        *_rows(outs[0], "k_out", d), *_rows(outs[1], "v_out", d), *_pages(k_cache, "k_cache", d),
        *_pages(v_cache, "v_cache", d), *scale_at, page_table.data_ptr(),
        0 if start is None else start.data_ptr(), cu.data_ptr(), tokens, num_pages, table_stride,
        hkv, d, _DT[dtype], codes, size, max_pages, B))
    return tuple(outs)


@functools.lru_cache(maxsize=256)
def _decode_need(B: int, hq: int, hkv: int, d: int) -> int:
    return _lib.load().rnn_attn_decode_q8_workspace_size(B, hq, hkv, d)


def attn_decode_q8(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   scales: torch.Tensor, page_table: torch.Tensor, lens: torch.Tensor, *,
                   scale: Optional[float] = None, with_lse: bool = False,
                   out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """``attn_decode`` over a cache of codes and scales: ``code * scale`` is attended to as it is.

    ``q [B, Hq, d]`` fp16 or bf16; all else is as in ``attn_decode``.
    """
    done = (_lib.fast or _lib.load_fast()).attn_decode_q8(
        q, k_cache, v_cache, scales, page_table, lens, scale, with_lse, out, workspace)
    if done is not None:
        return _lib.served(done, "rnn_attn_decode_q8")
    kind = _value_dtype(q, "q")
    dev = q.device
    _all(kind, dev, 3, q, "q")
    B, hq, d = q.shape
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache must be a [pages, page_size, heads, d] tensor")
    hkv = k_cache.shape[2]
    _heads(hq, hkv, d, _lib.RNN_ATTN_MAX_DIM)
    codes, _, num_pages, size, scale_at = _coded(k_cache, v_cache, scales, dev, hkv, d)
    _ints(lens, "lens", dev, B)
    table_stride, max_pages = _table(page_table, dev, B)
    scale = _scale(scale, d)
    out = _packed(q) if out is None else _given(out, q.shape, kind, dev, "out")
    lse = torch.empty((B, hq), dtype=torch.float32, device=dev) if with_lse else None
    if workspace is None:
        workspace = torch.empty(_decode_need(B, hq, hkv, d), dtype=torch.uint8, device=dev)
    ws, ws_bytes = _given_scratch(workspace, dev)
    _call(_lib.load().rnn_attn_decode_q8, "rnn_attn_decode_q8", q, _DECODE.pack(
        *_rows(q, "q", d), *_rows(out, "out", d), *_pages(k_cache, "k_cache", d),
        *_pages(v_cache, "v_cache", d), *scale_at, page_table.data_ptr(), lens.data_ptr(),
        0 if lse is None else lse.data_ptr(), ws, ws_bytes, num_pages, table_stride, size,
        max_pages, B, hq, hkv, d, _DT[kind], codes, scale))
    return (out, lse) if with_lse else out
