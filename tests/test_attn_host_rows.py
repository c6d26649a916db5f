"""Refusals of the attention entry points: outputs that cannot be written as they lie, and
keys without heads (no GPU: nothing is launched)."""
import ctypes
import itertools

import pytest
import torch

import reciprocal_nearest_neighbour_b200 as rnn
from reciprocal_nearest_neighbour_b200 import _lib, build as rnn_build
from test_attn_host import OnGpu

FAKE = 0x10000  # never dereferenced: every call below fails validation
EINVAL, EALIGN, EWS = 1, 2, 7
D = 64


@pytest.fixture(scope="module")
def lib():
    rnn_build.build()
    return _lib.load()


def rows(heads, p=FAKE, token=None, head=None):
    return _lib.Rows(p, heads * D if token is None else token, D if head is None else head)


PAGES = _lib.Pages(FAKE << 8, 16 * 2 * D, 2 * D, D)


def prompt(lib, out, tokens=10, heads=4, **kw):
    """EWS where nothing but the workspace is refused."""
    a = dict(q=rows(heads, FAKE << 4), k=rows(2, FAKE << 5), v=rows(2, FAKE << 6))
    a.update(kw)
    return lib.rnn_attn_prompt(ctypes.byref(_lib.AttnPromptArgs(
        q=a["q"], k=a["k"], v=a["v"], out=out, cu_q=FAKE, cu_k=FAKE, workspace=FAKE + 16,
        ws_bytes=256, Tq=tokens, Tk=10, Hq=heads, Hkv=2, d=D, dtype=0, B=1, causal=1,
        scale=0.1)), None)


def decode(lib, out, tokens=10, heads=4):
    return lib.rnn_attn_decode(ctypes.byref(_lib.AttnDecodeArgs(
        q=rows(heads, FAKE << 4), out=out, k_cache=PAGES, v_cache=PAGES, page_table=FAKE,
        lens=FAKE, num_pages=9, table_stride=5, page_size=16, max_pages=5, B=tokens, Hq=heads,
        Hkv=2, d=D, dtype=0, scale=0.1)), None)


def append(lib, q_out, tokens=10, heads=4, k_out=None, **kw):
    """EALIGN where nothing but the packed keys' address is refused."""
    a = dict(q=rows(heads, FAKE << 4), k=rows(2, FAKE << 5), v=rows(2, FAKE << 6))
    a.update(kw)
    return lib.rnn_kv_append(ctypes.byref(_lib.KvAppendArgs(
        q=a["q"], k=a["k"], v=a["v"], q_out=q_out,
        k_out=rows(2, FAKE + 2) if k_out is None else k_out, k_cache=PAGES, v_cache=PAGES,
        page_table=FAKE, start=FAKE, cu=FAKE, inv_freq=FAKE, T=tokens, num_pages=9,
        table_stride=5, Hq=heads, Hkv=2, d=D, dtype=0, page_size=16, max_pages=5, B=2, pairs=32,
        axes=1)), None)


def overlap(tokens, heads, token, head):
    at = sorted(t * token + h * head for t, h in itertools.product(range(tokens), range(heads)))
    return any(b - a < D for a, b in zip(at, at[1:]))


STRIDES = [D, D + 8, 2 * D, 2 * D + 8, 3 * D, 4 * D, 4 * D - 8, 5 * D, 8 * D, 9 * D + 16, 10 * D,
           11 * D - 8, 39 * D, 40 * D]


@pytest.mark.parametrize("tokens,heads", [(1, 4), (2, 2), (2, 4), (10, 4), (3, 8), (40, 2)])
def test_overlapping_rows_are_refused_and_no_others(lib, tokens, heads):
    """Against every pair of rows: nested strides, interleaved ones, and ones that meet late."""
    seen = set()
    for token, head in itertools.product(STRIDES, STRIDES):
        bad = overlap(tokens, heads, token if tokens > 1 else 0, head) if tokens > 1 else False
        seen.add(bad)
        out = rows(heads, token=token, head=head)
        assert prompt(lib, out, tokens, heads) == (EINVAL if bad else EWS), (token, head)
        assert decode(lib, out, tokens, heads) == (EINVAL if bad else EWS), (token, head)
        assert append(lib, out, tokens, heads) == (EINVAL if bad else EALIGN), (token, head)
    assert seen == ({False} if tokens == 1 else {False, True})


def test_overlapping_packed_keys_are_refused(lib):
    assert append(lib, rows(4), k_out=rows(2, token=D, head=D)) == EINVAL
    # queries are read only, and theirs may overlap
    assert prompt(lib, rows(4), q=rows(4, token=D, head=D)) == EWS


def test_outputs_in_place_of_other_inputs_are_refused(lib):
    q, k, v, q_out, k_out = (FAKE << n for n in (4, 5, 6, 8, 9))
    bad = [(k, k_out), (v, k_out), (q_out, v), (q_out, q), (q_out, q_out)]
    for at, ko in bad:
        assert append(lib, rows(4, at), k_out=rows(2, ko)) == EINVAL, (at, ko)
    # the cached values would be read after the keys had been turned in their place
    assert append(lib, rows(4, q_out), v=rows(2, k), k_out=rows(2, k)) == EINVAL
    for at in (k, v):
        assert lib.rnn_attn_prompt(ctypes.byref(_lib.AttnPromptArgs(
            q=rows(4, q), k=rows(2, k), v=rows(2, v), out=rows(4, at), cu_q=FAKE, cu_k=FAKE,
            Tq=10, Tk=10, Hq=4, Hkv=2, d=D, dtype=0, B=1, causal=1, scale=0.1)), None) == EINVAL


def test_append_without_key_heads_says_so():
    ints = dict(dtype=torch.int32)
    k, cache = OnGpu(8, 0, 64), OnGpu(5, 16, 0, 64)
    with pytest.raises(ValueError, match="no heads"):
        rnn.kv_append(k, k, cache, cache, OnGpu(2, 3, **ints), OnGpu(2, **ints), OnGpu(3, **ints))
