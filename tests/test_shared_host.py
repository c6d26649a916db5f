"""Refusals of the shared prefix's entry point (no GPU: nothing is launched)."""
import ctypes

import pytest
import torch

import reciprocal_nearest_neighbour_b200 as rnn
from reciprocal_nearest_neighbour_b200 import _lib, attn, build as rnn_build
from test_attn_host import FAKE, EALIGN, EINVAL, EUNSUP, EWS, OnGpu, pages, rows


@pytest.fixture(scope="module")
def lib():
    rnn_build.build()
    return _lib.load()


def test_packed_structure_matches(lib):
    kind, packed = _lib.AttnDecodeSharedArgs, attn._SHARED
    assert ctypes.sizeof(kind) == packed.size
    raw = (bytes(range(256)) * 3)[:packed.size]
    s = kind.from_buffer_copy(raw)
    mine = []
    for name, _ in kind._fields_:
        v = getattr(s, name)
        mine += [getattr(v, f) for f, _ in v._fields_] if hasattr(v, "_fields_") else [v]
    assert mine == list(packed.unpack(raw))


def test_errors(lib):
    size = lib.rnn_attn_decode_shared_workspace_size
    need = size(3, 4, 2, 64, 7 * 16)
    assert need > 0 and need % 256 == 0
    assert size(3, 4, 3, 64, 112) == 0 and size(-1, 4, 2, 64, 112) == 0 and size(3, 4, 2, 64, 0) == 0
    assert size(3, 4, 2, 136, 112) == 0
    assert size(0, 4, 2, 64, 112) > 0
    assert size(300, 4, 2, 64, 50000) > size(3, 4, 2, 64, 50000) > need

    def call(**kw):
        a = dict(q=rows(4), kc=pages(), vc=pages(), n=9, size=16, pp=FAKE, pl=FAKE, pn=7, table=FAKE,
                 ts=5, mp=5, lens=FAKE, B=3, hq=4, hkv=2, d=64, dt=1, scale=0.1,
                 out=rows(4, p=FAKE << 1), lse=None, ws=FAKE, wsn=need)
        a.update(kw)
        return lib.rnn_attn_decode_shared(ctypes.byref(_lib.AttnDecodeSharedArgs(
            q=a["q"], out=a["out"], k_cache=a["kc"], v_cache=a["vc"], prefix_pages=a["pp"],
            prefix_len=a["pl"], page_table=a["table"], lens=a["lens"], lse=a["lse"],
            workspace=a["ws"], ws_bytes=a["wsn"], num_pages=a["n"], table_stride=a["ts"],
            page_size=a["size"], prefix_pages_count=a["pn"], max_pages=a["mp"], B=a["B"],
            Hq=a["hq"], Hkv=a["hkv"], d=a["d"], dtype=a["dt"], scale=a["scale"])), None)

    assert lib.rnn_attn_decode_shared(None, None) == EINVAL
    assert call(B=-1) == EINVAL and call(n=0) == EINVAL and call(size=0) == EINVAL
    assert call(mp=0) == EINVAL and call(pn=0) == EINVAL and call(ts=-1) == EINVAL
    assert call(hq=5) == EINVAL and call(hkv=0) == EINVAL and call(dt=2) == EINVAL
    assert call(d=20) == EALIGN and call(hq=2048) == EUNSUP and call(B=1 << 30, ts=0) == EUNSUP
    for name in ("pp", "pl", "table", "lens"):
        assert call(**{name: None}) == EINVAL and call(**{name: FAKE + 2}) == EINVAL
    assert call(lse=FAKE + 1) == EINVAL
    for s in (0.0, -1.0, float("nan"), float("inf"), 2e38):
        assert call(scale=s) == EINVAL
    assert call(d=136, q=rows(4, 136), out=rows(4, 136), kc=pages(2, 136), vc=pages(2, 136)) == EUNSUP
    for name in ("kc", "vc"):
        assert call(**{name: pages(p=None)}) == EINVAL
        assert call(**{name: pages(p=FAKE + 8)}) == EALIGN
        assert call(**{name: pages(token=132)}) == EALIGN
        assert call(**{name: pages(page=8)}) == EINVAL
    assert call(q=rows(4, p=None)) == EINVAL and call(out=rows(4, head=3)) == EINVAL
    assert call(out=rows(4, p=FAKE << 1, token=128)) == EINVAL        # rows that overlap
    assert call(ws=None) == EWS and call(wsn=need - 1) == EWS and call(ws=FAKE + 128) == EWS
    assert call(pn=5000) == EWS                                       # a longer prefix needs more


def test_binding_checks_shapes_types_and_strides():
    I = dict(dtype=torch.int32)
    q, c = OnGpu(8, 4, 64), OnGpu(5, 16, 2, 64)
    pre, one, tab, lens = OnGpu(3, **I), OnGpu(1, **I), OnGpu(8, 3, **I), OnGpu(8, **I)
    bad = [
        (TypeError, (q.float(), c, c, pre, one, tab, lens)),
        (TypeError, (q, c.half(), c.half(), pre, one, tab, lens)),
        (ValueError, (q, c[0], c[0], pre, one, tab, lens)),
        (ValueError, (q, c, OnGpu(5, 8, 2, 64), pre, one, tab, lens)),
        (ValueError, (q, OnGpu(5, 16, 3, 64), OnGpu(5, 16, 3, 64), pre, one, tab, lens)),
        (ValueError, (q, c, c, OnGpu(0, **I), one, tab, lens)),
        (ValueError, (q, c, c, OnGpu(3, dtype=torch.int32, strides=(2,)), one, tab, lens)),
        (TypeError, (q, c, c, OnGpu(3, dtype=torch.int64), one, tab, lens)),
        (ValueError, (q, c, c, pre, OnGpu(2, **I), tab, lens)),
        (TypeError, (q, c, c, pre, OnGpu(1, dtype=torch.int64), tab, lens)),
        (ValueError, (q, c, c, pre, 640, tab, lens)),
        (ValueError, (q, c, c, pre, one, OnGpu(7, 3, **I), lens)),
        (ValueError, (q, c, c, pre, one, tab, OnGpu(9, **I))),
        (ValueError, (OnGpu(8, 4, 136), OnGpu(5, 16, 2, 136), OnGpu(5, 16, 2, 136), pre, one, tab, lens)),
    ]
    for err, args in bad:
        with pytest.raises(err):
            rnn.attn_decode_shared(*args)
    for kw in (dict(scale=0.0), dict(out=OnGpu(8, 2, 64)), dict(workspace=OnGpu(8))):
        with pytest.raises(ValueError):
            rnn.attn_decode_shared(q, c, c, pre, one, tab, lens, **kw)
    x, k = torch.zeros((4, 2, 64), dtype=torch.bfloat16), torch.zeros((2, 16, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        rnn.attn_decode_shared(x, k, k, i, i[:1], torch.zeros((4, 2), dtype=torch.int32), i)
