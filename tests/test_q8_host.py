"""Refusals of the 8-bit cache's entry points (no GPU: nothing is launched)."""
import ctypes

import pytest
import torch

import reciprocal_nearest_neighbour_b200 as rnn
from reciprocal_nearest_neighbour_b200 import _lib, build as rnn_build, cache_q8
from test_attn_host import FAKE, EALIGN, EINVAL, EUNSUP, EWS, OnGpu, pages, rows

E4 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def lib():
    rnn_build.build()
    return _lib.load()


def scales(heads=2, size=16, p=FAKE, page=None, head=None):
    return _lib.Scales(p, 2 * size * heads if page is None else page,
                       2 * size if head is None else head)


def test_packed_structures_match(lib):
    for kind, packed in ((_lib.KvAppendQ8Args, cache_q8._APPEND), (_lib.KvReadQ8Args, cache_q8._READ),
                         (_lib.AttnDecodeQ8Args, cache_q8._DECODE)):
        assert ctypes.sizeof(kind) == packed.size
        raw = (bytes(range(256)) * 3)[:packed.size]
        s = kind.from_buffer_copy(raw)
        mine = []
        for name, _ in kind._fields_:
            v = getattr(s, name)
            mine += [getattr(v, f) for f, _ in v._fields_] if hasattr(v, "_fields_") else [v]
        assert mine == list(packed.unpack(raw))


def cache_errors(call):
    """What every call with a cache of codes refuses."""
    assert call(codes=2) == EINVAL and call(codes=-1) == EINVAL and call(dt=2) == EINVAL
    assert call(n=0) == EINVAL and call(size=0) == EINVAL and call(mp=0) == EINVAL
    assert call(ts=-1) == EINVAL and call(d=0) == EINVAL and call(d=20) == EALIGN
    assert call(hkv=0) == EINVAL and call(B=-1) == EINVAL and call(table=None) == EINVAL
    for name in ("kc", "vc"):
        assert call(**{name: pages(p=None)}) == EINVAL
        assert call(**{name: pages(p=FAKE + 8)}) == EALIGN
        assert call(**{name: pages(head=70)}) == EALIGN
        assert call(**{name: pages(token=8)}) == EINVAL
    assert call(sc=scales(p=None)) == EINVAL and call(sc=scales(p=FAKE + 4)) == EINVAL
    assert call(sc=scales(head=30)) == EINVAL and call(sc=scales(page=2)) == EINVAL
    assert call(sc=scales(head=33)) == EALIGN and call(sc=scales(page=131)) == EALIGN
    # strides beyond 32-bit numbers of 8 codes, or of pairs of scales
    for name in ("kc", "vc"):
        assert call(**{name: pages(page=1 << 34)}) == EUNSUP
        assert call(**{name: pages(head=1 << 34)}) == EUNSUP
    assert call(sc=scales(page=1 << 32)) == EUNSUP and call(sc=scales(head=1 << 32)) == EUNSUP


def test_append_errors(lib):
    def call(**kw):
        a = dict(q=rows(4), k=rows(p=FAKE << 1), v=rows(p=FAKE << 2), T=10, hq=4, hkv=2, d=64, dt=0,
                 codes=0, kc=pages(), vc=pages(), sc=scales(), n=9, size=16, table=FAKE, ts=5, mp=5,
                 start=FAKE, cu=FAKE, B=2, pos=None, ps=0, inv=FAKE, pairs=32, axes=1,
                 qo=rows(4, p=FAKE << 3), ko=_lib.Rows(None, 0, 0))
        a.update(kw)
        return lib.rnn_kv_append_q8(ctypes.byref(_lib.KvAppendQ8Args(
            q=a["q"], k=a["k"], v=a["v"], q_out=a["qo"], k_out=a["ko"], k_cache=a["kc"],
            v_cache=a["vc"], scales=a["sc"], page_table=a["table"], start=a["start"], cu=a["cu"],
            positions=a["pos"], inv_freq=a["inv"], T=a["T"], num_pages=a["n"],
            table_stride=a["ts"], position_stride=a["ps"], Hq=a["hq"], Hkv=a["hkv"], d=a["d"],
            dtype=a["dt"], codes=a["codes"], page_size=a["size"], max_pages=a["mp"], B=a["B"],
            pairs=a["pairs"], axes=a["axes"])), None)

    assert lib.rnn_kv_append_q8(None, None) == EINVAL
    cache_errors(call)
    assert call(T=-1) == EINVAL and call(hq=-1) == EINVAL and call(cu=FAKE + 1) == EINVAL
    assert call(d=264, pairs=0, axes=0) == EUNSUP and call(hq=2048) == EUNSUP
    assert call(pairs=33) == EINVAL and call(pairs=0) == EINVAL and call(axes=0) == EINVAL
    assert call(axes=3, pairs=8) == EINVAL and call(inv=None) == EINVAL
    assert call(inv=FAKE + 4) == EINVAL and call(axes=2, pairs=16) == EINVAL
    assert call(axes=2, pairs=16, pos=FAKE, ps=1) == EINVAL and call(start=None) == EINVAL
    for name, h in (("q", 4), ("k", 2), ("v", 2), ("qo", 4), ("ko", 2)):
        assert call(**{name: rows(h, p=FAKE + 2)}) == EALIGN
        assert call(**{name: rows(h, token=8)}) == EINVAL
    # outputs in the place of other inputs, or of their own with other strides
    assert call(qo=rows(4, p=FAKE << 1)) == EINVAL and call(qo=rows(4, p=FAKE << 2)) == EINVAL
    assert call(ko=rows(p=FAKE)) == EINVAL and call(ko=rows(p=FAKE << 2)) == EINVAL
    assert call(ko=rows(p=FAKE << 3)) == EINVAL
    assert call(qo=rows(4, token=512)) == EINVAL and call(ko=rows(p=FAKE << 1, token=256)) == EINVAL
    assert call(qo=rows(4, p=FAKE << 3, token=32 * 6)) == EINVAL      # rows that overlap


def test_read_errors(lib):
    def call(**kw):
        a = dict(k=rows(p=FAKE << 1), v=rows(p=FAKE << 2), T=10, hkv=2, d=64, dt=0, codes=0,
                 kc=pages(), vc=pages(), sc=scales(), n=9, size=16, table=FAKE, ts=5, mp=5,
                 start=None, cu=FAKE, B=2)
        a.update(kw)
        return lib.rnn_kv_read_q8(ctypes.byref(_lib.KvReadQ8Args(
            k=a["k"], v=a["v"], k_cache=a["kc"], v_cache=a["vc"], scales=a["sc"],
            page_table=a["table"], start=a["start"], cu=a["cu"], T=a["T"], num_pages=a["n"],
            table_stride=a["ts"], Hkv=a["hkv"], d=a["d"], dtype=a["dt"], codes=a["codes"],
            page_size=a["size"], max_pages=a["mp"], B=a["B"])), None)

    assert lib.rnn_kv_read_q8(None, None) == EINVAL
    cache_errors(call)
    assert call(T=-1) == EINVAL and call(start=FAKE + 2) == EINVAL and call(cu=None) == EINVAL
    assert call(d=264) == EUNSUP and call(hkv=2048) == EUNSUP
    assert call(k=rows(p=None)) == EINVAL and call(v=rows(p=FAKE + 8)) == EALIGN
    assert call(k=rows(p=FAKE << 2)) == EINVAL and call(v=rows(token=96)) == EINVAL


def test_decode_errors(lib):
    need = lib.rnn_attn_decode_q8_workspace_size(3, 4, 2, 64)
    assert need > 0 and need % 256 == 0
    assert lib.rnn_attn_decode_q8_workspace_size(3, 4, 3, 64) == 0

    def call(**kw):
        a = dict(q=rows(4), kc=pages(), vc=pages(), sc=scales(), n=9, size=16, table=FAKE, ts=5,
                 mp=5, lens=FAKE, B=3, hq=4, hkv=2, d=64, dt=1, codes=1, scale=0.1,
                 out=rows(4, p=FAKE << 1), lse=None, ws=FAKE, wsn=need)
        a.update(kw)
        return lib.rnn_attn_decode_q8(ctypes.byref(_lib.AttnDecodeQ8Args(
            q=a["q"], out=a["out"], k_cache=a["kc"], v_cache=a["vc"], scales=a["sc"],
            page_table=a["table"], lens=a["lens"], lse=a["lse"], workspace=a["ws"],
            ws_bytes=a["wsn"], num_pages=a["n"], table_stride=a["ts"], page_size=a["size"],
            max_pages=a["mp"], B=a["B"], Hq=a["hq"], Hkv=a["hkv"], d=a["d"], dtype=a["dt"],
            codes=a["codes"], scale=a["scale"])), None)

    assert lib.rnn_attn_decode_q8(None, None) == EINVAL
    cache_errors(call)
    assert call(hq=5) == EINVAL and call(lens=FAKE + 3) == EINVAL and call(lse=FAKE + 2) == EINVAL
    for s in (0.0, -1.0, float("nan"), float("inf"), 2e38):
        assert call(scale=s) == EINVAL
    assert call(d=136, q=rows(4, 136), out=rows(4, 136), kc=pages(2, 136),
                vc=pages(2, 136)) == EUNSUP
    assert call(B=1 << 30, ts=0) == EUNSUP
    assert call(q=rows(4, p=None)) == EINVAL and call(out=rows(4, head=3)) == EINVAL
    assert call(ws=None) == EWS and call(wsn=need - 1) == EWS and call(ws=FAKE + 128) == EWS


def test_binding_checks_shapes_types_and_strides():
    I, F = dict(dtype=torch.int32), dict(dtype=torch.float32)
    q, k, c = OnGpu(8, 4, 64), OnGpu(8, 2, 64), OnGpu(5, 16, 2, 64, dtype=E4)
    c8 = OnGpu(5, 16, 2, 64, dtype=torch.int8)
    s, tab, lens, cu = OnGpu(5, 2, 16, 2, **F), OnGpu(8, 3, **I), OnGpu(8, **I), OnGpu(3, **I)
    bad = [
        (TypeError, (q.float(), c, c, s, tab, lens)),
        (TypeError, (q, k.view(2, 4, 2, 64), c, s, tab, lens)),      # a cache of values
        (TypeError, (q, c, c8, s, tab, lens)),                       # two kinds of codes
        (ValueError, (q, c[0], c[0], s, tab, lens)),
        (ValueError, (q, c, OnGpu(5, 8, 2, 64, dtype=E4), s, tab, lens)),
        (ValueError, (q, OnGpu(5, 16, 2, 32, dtype=E4), OnGpu(5, 16, 2, 32, dtype=E4), s, tab, lens)),
        (ValueError, (q, c, c, OnGpu(5, 16, 2, 2, **F), tab, lens)),  # rows and heads swapped
        (TypeError, (q, c, c, OnGpu(5, 2, 16, 2, dtype=torch.float16), tab, lens)),
        (ValueError, (q, c, c, OnGpu(5, 2, 16, 2, strides=(64, 32, 1, 16), **F), tab, lens)),
        (ValueError, (q, c, c, OnGpu(5, 2, 16, 2, strides=(64, 31, 2, 1), **F), tab, lens)),
        (ValueError, (q, c, c, OnGpu(5, 2, 16, 2, strides=(65, 32, 2, 1), **F), tab, lens)),
        (ValueError, (q, c, c, s, OnGpu(7, 3, **I), lens)),
        (ValueError, (q, c, c, s, tab, OnGpu(9, **I))),
        (ValueError, (OnGpu(8, 4, 136), OnGpu(5, 16, 2, 136, dtype=E4),
                      OnGpu(5, 16, 2, 136, dtype=E4), s, tab, lens)),
        (ValueError, (q, OnGpu(5, 16, 2, 64, dtype=E4, strides=(2048, 128, 68, 1)), c, s, tab, lens)),
    ]
    for err, args in bad:
        with pytest.raises(err):
            rnn.attn_decode_q8(*args)
    with pytest.raises(ValueError):
        rnn.attn_decode_q8(q, c, c, s, tab, lens, scale=0.0)
    with pytest.raises(ValueError):
        rnn.attn_decode_q8(q, c, c, s, tab, lens, out=k)
    tab, start = OnGpu(2, 3, **I), OnGpu(2, **I)
    ok = (k, k, c, c, s, tab, start, cu)
    inv = OnGpu(32, dtype=torch.float64)
    bad = [
        (ValueError, ok, dict(q=q)),                                      # nothing to rotate by
        (ValueError, ok, dict(q_out=q)),
        (ValueError, ok, dict(inv_freq=OnGpu(33, dtype=torch.float64))),
        (ValueError, ok, dict(positions=OnGpu(8, **I))),
        (ValueError, ok, dict(inv_freq=inv, positions=OnGpu(8, 3, **I))),
        (ValueError, ok, dict(inv_freq=inv, q=OnGpu(7, 4, 64))),
        (ValueError, ok, dict(k_out=OnGpu(8, 4, 64))),
        (TypeError, (k, k, c8, c, s, tab, start, cu), {}),
        (ValueError, (k, k, c, c, s, tab, OnGpu(3, **I), cu), {}),
        (ValueError, (k, k, OnGpu(5, 16, 3, 64, dtype=E4), OnGpu(5, 16, 3, 64, dtype=E4), s, tab,
                      start, cu), {}),
    ]
    for err, args, kw in bad:
        with pytest.raises(err):
            rnn.kv_append_q8(*args, **kw)
    bad = [
        (TypeError, (c, c, s, tab, cu, 8, torch.float32), {}),
        (ValueError, (c, c, s, tab, cu, -1), {}),
        (ValueError, (c, c, s, tab, OnGpu(4, **I), 8), {}),
        (ValueError, (c, c, s, tab, cu, 8), dict(start=OnGpu(3, **I))),
        (ValueError, (c, c, s, tab, cu, 8), dict(k_out=OnGpu(9, 2, 64))),
        (TypeError, (c, c, s, tab, cu, 8), dict(v_out=OnGpu(8, 2, 64, dtype=torch.float16))),
        (TypeError, (k, k, s, tab, cu, 8), {}) if k.dim() == 4 else (ValueError, (k, k, s, tab, cu, 8), {}),
    ]
    for err, args, kw in bad:
        with pytest.raises(err):
            rnn.kv_read_q8(*args, **kw)


def test_binding_refuses_cpu_tensors():
    c, s = torch.zeros((2, 16, 2, 64), dtype=torch.int8), torch.zeros((2, 2, 16, 2))
    i = torch.zeros(2, dtype=torch.int32)
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        rnn.attn_decode_q8(x, c, c, s, torch.zeros((4, 2), dtype=torch.int32), i)
    with pytest.raises(ValueError):
        rnn.kv_append_q8(x, x, c, c, s, torch.zeros((1, 2), dtype=torch.int32), i[:1], i)
    with pytest.raises(ValueError):
        rnn.kv_read_q8(c, c, s, torch.zeros((1, 2), dtype=torch.int32), i, 4)


def test_extension_module_serves_no_unusual_call(lib):
    """What is not as expected comes back as None, for the Python form to look at."""
    fast = _lib.load_fast()
    assert fast.__name__.endswith("_fast")
    for name, n in (("attn_decode_q8", 10), ("attn_decode_shared", 11), ("kv_read_q8", 10),
                    ("kv_append_q8", 15)):
        call = getattr(fast, name)
        assert call() is None and call(*[None] * n) is None and call(*[1.5] * n) is None
        assert call(*[torch.zeros(2, 2, 64, dtype=torch.float16)] * n) is None
        assert call(*[OnGpu(2, 2, 64)] * n) is None
    with pytest.raises(TypeError):
        fast.bind(1, 2)
    with pytest.raises(ValueError):
        fast.bind(0, 0, 0, 0, 0, 0)
