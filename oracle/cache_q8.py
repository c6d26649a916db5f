"""The 8-bit cache in double precision (numpy): codes, scales and their values.

Test infrastructure for ``kv_append_q8``, ``kv_read_q8`` and ``attn_decode_q8``:
written from the formulas, and sharing no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np

TOP = {"e4m3": 448.0, "int8": 127.0}


def e4m3_value(code):
    """Values of e4m3 codes (bytes): sign, 4 bits of exponent with bias 7, 3 of mantissa."""
    code = np.asarray(code, dtype=np.int64)
    sign = np.where(code & 128, -1.0, 1.0)
    exp, man = (code >> 3) & 15, code & 7
    x = np.where(exp == 0, man * 2.0 ** -9, (8 + man) * 2.0 ** (exp - 10.0))
    return np.where((code & 127) == 127, np.nan, sign * x)


def value(code, codes):
    """Values of codes given as bytes."""
    code = np.asarray(code, dtype=np.uint8)
    return e4m3_value(code) if codes == "e4m3" else code.view(np.int8).astype(np.float64)


def half_step(x, codes):
    """Largest distance of a rounded code from ``x``, a row in units of its scale."""
    if codes == "int8":
        return np.full_like(x, 0.5)
    return 2.0 ** (np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6))) - 4)


def scale(x, codes):
    """Scales of rows ``x [..., d]``."""
    return np.maximum(np.abs(x).max(-1) / TOP[codes], 2.0 ** -126)


def nearest_e4m3(x):
    """e4m3 values nearest to ``x`` (|x| <= 448), ties to the even code."""
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6))) - 3)
    return np.rint(x / step) * step


def quantise32(x, codes):
    """Code values and scales of fp32 rows, with fp32's own quotients."""
    x = np.asarray(x, dtype=np.float32)
    s = np.maximum(np.abs(x).max(-1) / np.float32(TOP[codes]), np.float32(2.0 ** -126))
    y = (x * (np.float32(1) / s)[..., None]).astype(np.float64)
    return (nearest_e4m3(y) if codes == "e4m3" else np.rint(y)), s
