"""Pins of the shared prefix's oracle against attention over one page table."""
import numpy as np

from oracle import attention as oa
from oracle.shared import decode_shared


def test_prefix_of_whole_pages_is_a_longer_table():
    rng = np.random.default_rng(0)
    k, v = (rng.normal(size=(9, 4, 2, 8)) for _ in range(2))
    q = rng.normal(size=(3, 4, 8))
    prefix, table, lens = [5, 2], np.array([[0, 1], [8, 3], [6, 7]]), [5, 1, 8]
    got = decode_shared(q, k, v, prefix, 8, table, lens, 0.3)
    want = oa.decode(q, k, v, np.hstack([np.tile(prefix, (3, 1)), table]), [8 + n for n in lens], 0.3)
    for f in ("out", "lse", "spread", "reach", "keys"):
        assert np.array_equal(getattr(got, f), getattr(want, f))


def test_empty_sides():
    rng = np.random.default_rng(1)
    k, v = (rng.normal(size=(4, 4, 1, 8)) for _ in range(2))
    q = rng.normal(size=(2, 1, 8))
    table = np.array([[1], [2]])
    own = decode_shared(q, k, v, [0], 0, table, [3, 0], 1.0)
    want = oa.decode(q, k, v, table, [3, 0], 1.0)
    assert np.array_equal(own.out, want.out) and own.keys[1, 0] == 0 and np.isneginf(own.lse[1, 0])
    only = decode_shared(q, k, v, [0], 3, table, [0, 0], 1.0)
    want = oa.decode(q, k, v, np.array([[0], [0]]), [3, 3], 1.0)
    assert np.array_equal(only.out, want.out)
    # a page that does not exist takes its rows with it
    part = decode_shared(q, k, v, [-1, 3], 6, table, [0, 0], 1.0)
    want = oa.decode(q, k, v, np.array([[3], [3]]), [2, 2], 1.0)
    assert np.array_equal(part.out, want.out)
