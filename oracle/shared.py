"""Attention over a shared prefix and each sequence's own tokens, in double precision.

Test infrastructure for ``attn_decode_shared``.
"""
from __future__ import annotations

import numpy as np

from .attention import Attn, _empty, _row


def decode_shared(q, k_cache, v_cache, prefix_pages, prefix_len, table, lens, scale) -> Attn:
    """One row per sequence over the rows of the prefix and its own whose page exists."""
    q = np.asarray(q, dtype=np.float64)
    pages, size, hkv = k_cache.shape[:3]
    group = q.shape[1] // hkv
    r = _empty(*q.shape)

    def rows_of(names, n):
        t = np.arange(min(max(int(n), 0), len(names) * size))
        page = np.asarray(names)[t // size]
        there = (page >= 0) & (page < pages)
        return page[there], t[there] % size

    ahead = rows_of(prefix_pages, prefix_len)
    for b in range(q.shape[0]):
        page, row = (np.concatenate(x) for x in zip(ahead, rows_of(table[b], lens[b])))
        if not len(page):
            continue
        K = np.asarray(k_cache[page, row], dtype=np.float64)
        V = np.asarray(v_cache[page, row], dtype=np.float64)
        for h in range(q.shape[1]):
            r.out[b, h], r.lse[b, h], r.spread[b, h], r.reach[b, h] = _row(
                q[b, h], K[:, h // group], V[:, h // group], scale)
            r.keys[b, h] = len(page)
    return r
