"""Attention in double precision (numpy), one sequence and head at a time.

Test infrastructure for ``kv_append``, ``attn_prompt`` and ``attn_decode``:
written from the formulas, and sharing no code with the CUDA path.  Beside the
results it returns what the error bounds of the tests are made of.
"""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np


@dataclass
class Attn:
    out: np.ndarray      # [rows, heads, d]
    lse: np.ndarray      # [rows, heads]
    spread: np.ndarray   # [rows, heads, d]: the weighted sum of |v|
    reach: np.ndarray    # [rows, heads]: largest scale * sum |q_c k_c| over the keys seen
    keys: np.ndarray     # [rows, heads]: number of keys seen


def _empty(rows, heads, d):
    return Attn(np.zeros((rows, heads, d)), np.full((rows, heads), -np.inf),
                np.zeros((rows, heads, d)), np.zeros((rows, heads)), np.zeros((rows, heads), int))


def _row(q, K, V, scale):
    """One query over its keys: softmax(scale K q)-weighted sum of V."""
    s = scale * (K @ q)
    w = np.exp(s - s.max())
    total = w.sum()
    return (w @ V) / total, s.max() + np.log(total), (w @ np.abs(V)) / total, \
        scale * (np.abs(K) @ np.abs(q)).max()


def prompt(q, k, v, cu_q, cu_k, causal, scale) -> Attn:
    """Packed sequences; rows outside them keep zeros (and -inf)."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    group = q.shape[1] // k.shape[1]
    r = _empty(*q.shape)
    for b in range(len(cu_q) - 1):
        nq, nk = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        for i in range(nq):
            seen = min(nk, i + nk - nq + 1) if causal else nk
            if seen <= 0:
                continue
            at, ks = cu_q[b] + i, slice(cu_k[b], cu_k[b] + seen)
            for h in range(q.shape[1]):
                r.out[at, h], r.lse[at, h], r.spread[at, h], r.reach[at, h] = _row(
                    q[at, h], k[ks, h // group], v[ks, h // group], scale)
                r.keys[at, h] = seen
    return r


def decode(q, k_cache, v_cache, table, lens, scale) -> Attn:
    """One row per sequence over the cached rows whose page exists."""
    q = np.asarray(q, dtype=np.float64)
    pages, size, hkv = k_cache.shape[:3]
    group = q.shape[1] // hkv
    r = _empty(*q.shape)
    for b in range(q.shape[0]):
        t = np.arange(min(max(int(lens[b]), 0), table.shape[1] * size))
        page = np.asarray(table[b])[t // size]
        there = (page >= 0) & (page < pages)
        if not there.any():
            continue
        K = np.asarray(k_cache[page[there], t[there] % size], dtype=np.float64)
        V = np.asarray(v_cache[page[there], t[there] % size], dtype=np.float64)
        for h in range(q.shape[1]):
            r.out[b, h], r.lse[b, h], r.spread[b, h], r.reach[b, h] = _row(
                q[b, h], K[:, h // group], V[:, h // group], scale)
            r.keys[b, h] = there.sum()
    return r


def rotate(x, positions, inv_freq, paired):
    """``x [T, H, d]`` turned by ``positions [T, axes] * inv_freq [pairs]``."""
    x = np.array(x, dtype=np.float64)
    pairs = len(inv_freq)
    for t in range(x.shape[0]):
        for a in range(positions.shape[1]):
            for i in range(pairs):
                one = 2 * pairs * a + (2 * i if paired else i)
                two = one + (1 if paired else pairs)
                angle = float(positions[t, a]) * float(inv_freq[i])
                c, s = np.cos(angle), np.sin(angle)
                x1, x2 = x[t, :, one].copy(), x[t, :, two].copy()
                x[t, :, one], x[t, :, two] = x1 * c - x2 * s, x2 * c + x1 * s
    return x


def slots(cu, start, table, size, pages, T):
    """Per token (page, row) in the cache, or None where it is not stored; and its number."""
    where, number = [None] * T, [None] * T
    for b in range(len(cu) - 1):
        for t in range(cu[b], cu[b + 1]):
            n = int(start[b]) + t - cu[b]
            number[t] = n
            if 0 <= n < table.shape[1] * size and 0 <= table[b][n // size] < pages:
                where[t] = (int(table[b][n // size]), n % size)
    return where, number
