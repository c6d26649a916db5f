"""Pins of the double-precision attention oracle (CPU)."""
import math

import numpy as np
import pytest

from oracle import attention as oa


def test_two_keys_by_hand():
    # scores 0 and ln 3: weights 1/4 and 3/4
    q = np.array([[[1.0, 0.0]]])
    k = np.array([[[0.0, 5.0]], [[math.log(3.0), 1.0]]])
    v = np.array([[[4.0, 0.0]], [[8.0, -4.0]]])
    r = oa.prompt(q, k, v, [0, 1], [0, 2], True, 1.0)
    assert np.allclose(r.out[0, 0], [7.0, -3.0], atol=1e-15)
    assert np.isclose(r.lse[0, 0], math.log(4.0))
    assert np.allclose(r.spread[0, 0], [7.0, 3.0]) and r.keys[0, 0] == 2


def test_causal_rows_and_empty_rows():
    rng = np.random.default_rng(0)
    q, k, v = (rng.standard_normal((n, 1, 4)) for n in (5, 3, 3))
    r = oa.prompt(q, k, v, [0, 5], [0, 3], True, 0.5)
    # the last query sees the last key; the first two see nothing
    assert r.keys[:, 0].tolist() == [0, 0, 1, 2, 3]
    assert np.all(r.out[:2] == 0) and np.all(np.isneginf(r.lse[:2]))
    assert np.allclose(r.out[2], v[0])
    full = oa.prompt(q, k, v, [0, 5], [0, 3], False, 0.5)
    assert np.allclose(full.out[4], r.out[4]) and full.keys.min() == 3


def test_grouped_heads_read_their_key_head():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((3, 4, 8)), rng.standard_normal((3, 2, 8)), \
        rng.standard_normal((3, 2, 8))
    r = oa.prompt(q, k, v, [0, 3], [0, 3], False, 1.0)
    for h in range(4):
        one = oa.prompt(q[:, h:h + 1], k[:, h // 2:h // 2 + 1], v[:, h // 2:h // 2 + 1], [0, 3],
                        [0, 3], False, 1.0)
        assert np.allclose(one.out[:, 0], r.out[:, h])


def test_decode_equals_the_last_prompt_row():
    rng = np.random.default_rng(2)
    n, size = 11, 4
    q, k, v = (rng.standard_normal((n, 2, 8)) for _ in range(3))
    table = np.array([[5, 0, 3]])
    kc, vc = np.full((6, size, 2, 8), np.nan), np.full((6, size, 2, 8), np.nan)
    where, number = oa.slots([0, n], [0], table, size, 6, n)
    assert where[0] == (5, 0) and where[4] == (0, 0) and where[10] == (3, 2)
    assert number == list(range(n))
    for t, (p, row) in enumerate(where):
        kc[p, row], vc[p, row] = k[t], v[t]
    r = oa.prompt(q, k, v, [0, n], [0, n], True, 0.3)
    d = oa.decode(q[-1:], kc, vc, table, [n], 0.3)
    assert np.allclose(d.out[0], r.out[-1]) and np.allclose(d.lse[0], r.lse[-1])
    # keys on a page that does not exist are absent
    gone = oa.decode(q[-1:], kc, vc, np.array([[5, -1, 3]]), [n], 0.3)
    keep = [0, 1, 2, 3, 8, 9, 10]
    part = oa.prompt(q[-1:], k[keep], v[keep], [0, 1], [0, 7], False, 0.3)
    assert np.allclose(gone.out[0], part.out[0]) and gone.keys[0, 0] == 7


@pytest.mark.parametrize("paired", [False, True])
def test_rotation(paired):
    # a quarter turn swaps the pair; relative angles survive in dot products
    x = np.arange(1.0, 9.0).reshape(1, 1, 8)
    y = oa.rotate(x, np.array([[1]]), [math.pi / 2, 0.0], paired)
    if paired:
        assert np.allclose(y[0, 0], [-2, 1, 3, 4, 5, 6, 7, 8])
    else:
        assert np.allclose(y[0, 0], [-3, 2, 1, 4, 5, 6, 7, 8])
    rng = np.random.default_rng(3)
    a, b, f = rng.standard_normal((1, 1, 8)), rng.standard_normal((1, 1, 8)), [1.0, 0.1]
    pos = lambda i, j: np.array([[i, j]])
    dot = lambda i, j: float(np.sum(oa.rotate(a, pos(7 + i, 2 + j), f, paired) *
                                    oa.rotate(b, pos(3 + i, 9 + j), f, paired)))
    assert np.isclose(dot(0, 0), dot(100, 31))
