"""Refusals of the attention entry points (no GPU: nothing is launched)."""
import ctypes

import pytest
import torch

import reciprocal_nearest_neighbour_b200 as rnn
from reciprocal_nearest_neighbour_b200 import _lib, build as rnn_build

FAKE = 0x10000  # never dereferenced: every call below fails validation first
EINVAL, EALIGN, EUNSUP, EWS = 1, 2, 6, 7


@pytest.fixture(scope="module")
def lib():
    rnn_build.build()
    return _lib.load()


def rows(heads=2, d=64, p=FAKE, token=None, head=None):
    return _lib.Rows(p, heads * d if token is None else token, d if head is None else head)


def pages(heads=2, d=64, size=16, p=FAKE, page=None, token=None, head=None):
    return _lib.Pages(p, size * heads * d if page is None else page,
                      heads * d if token is None else token, d if head is None else head)


def test_packed_structures_match(lib):
    from reciprocal_nearest_neighbour_b200 import attn

    for kind, packed in ((_lib.KvAppendArgs, attn._APPEND), (_lib.AttnPromptArgs, attn._PROMPT),
                         (_lib.AttnDecodeArgs, attn._DECODE)):
        assert ctypes.sizeof(kind) == packed.size
        raw = (bytes(range(256)) * 2)[:packed.size]
        flat = packed.unpack(raw)
        s = kind.from_buffer_copy(raw)
        mine = []
        for name, _ in kind._fields_:
            v = getattr(s, name)
            mine += [getattr(v, f) for f, _ in v._fields_] if hasattr(v, "_fields_") else [v]
        assert mine == list(flat)


def test_prompt_errors(lib):
    need = lib.rnn_attn_prompt_workspace_size()

    def call(**kw):
        a = dict(q=rows(4), k=rows(), v=rows(), tq=10, tk=10, hq=4, hkv=2, d=64, dt=0, cq=FAKE,
                 ck=FAKE, B=1, causal=1, scale=0.1, out=rows(4), lse=None, ws=FAKE, n=need)
        a.update(kw)
        return lib.rnn_attn_prompt(ctypes.byref(_lib.AttnPromptArgs(
            q=a["q"], k=a["k"], v=a["v"], out=a["out"], cu_q=a["cq"], cu_k=a["ck"], lse=a["lse"],
            workspace=a["ws"], ws_bytes=a["n"], Tq=a["tq"], Tk=a["tk"], Hq=a["hq"], Hkv=a["hkv"],
            d=a["d"], dtype=a["dt"], B=a["B"], causal=a["causal"], scale=a["scale"])), None)

    assert lib.rnn_attn_prompt(None, None) == EINVAL

    assert call(tq=-1) == EINVAL and call(B=-1) == EINVAL and call(tk=1 << 31) == EINVAL
    assert call(hq=0) == EINVAL and call(hq=3) == EINVAL and call(hkv=0) == EINVAL
    assert call(dt=2) == EINVAL and call(d=0) == EINVAL
    assert call(d=20) == EALIGN and call(d=136, q=rows(4, 136), out=rows(4, 136),
                                         k=rows(2, 136), v=rows(2, 136)) == EUNSUP
    assert call(hq=2048) == EUNSUP
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=s) == EINVAL
    assert call(cq=None) == EINVAL and call(ck=FAKE + 2) == EINVAL and call(lse=FAKE + 1) == EINVAL
    for name in ("q", "k", "v", "out"):
        h = 4 if name in ("q", "out") else 2
        assert call(**{name: rows(h, p=None)}) == EINVAL
        assert call(**{name: rows(h, p=FAKE + 8)}) == EALIGN
        assert call(**{name: rows(h, token=260)}) == EALIGN
        assert call(**{name: rows(h, head=68)}) == EALIGN
        assert call(**{name: rows(h, head=0)}) == EINVAL
    assert call(ws=FAKE + 16) == EWS and call(n=need - 1) == EWS


def test_decode_errors(lib):
    need = lib.rnn_attn_decode_workspace_size(3, 4, 2, 64)
    assert need > 0 and need % 256 == 0
    assert lib.rnn_attn_decode_workspace_size(3, 4, 3, 64) == 0
    assert lib.rnn_attn_decode_workspace_size(-1, 4, 2, 64) == 0

    def call(**kw):
        a = dict(q=rows(4), k=pages(), v=pages(), n=9, size=16, table=FAKE, ts=5, mp=5, lens=FAKE,
                 B=3, hq=4, hkv=2, d=64, dt=1, scale=0.1, out=rows(4), lse=None, ws=FAKE,
                 wsn=need)
        a.update(kw)
        return lib.rnn_attn_decode(ctypes.byref(_lib.AttnDecodeArgs(
            q=a["q"], out=a["out"], k_cache=a["k"], v_cache=a["v"], page_table=a["table"],
            lens=a["lens"], lse=a["lse"], workspace=a["ws"], ws_bytes=a["wsn"], num_pages=a["n"],
            table_stride=a["ts"], page_size=a["size"], max_pages=a["mp"], B=a["B"], Hq=a["hq"],
            Hkv=a["hkv"], d=a["d"], dtype=a["dt"], scale=a["scale"])), None)

    assert lib.rnn_attn_decode(None, None) == EINVAL

    assert call(B=-1) == EINVAL and call(n=0) == EINVAL and call(size=0) == EINVAL
    assert call(mp=0) == EINVAL and call(ts=-1) == EINVAL and call(hq=5) == EINVAL
    assert call(table=None) == EINVAL and call(lens=FAKE + 3) == EINVAL and call(dt=9) == EINVAL
    assert call(scale=0.0) == EINVAL and call(d=12) == EALIGN
    assert call(d=136, q=rows(4, 136), out=rows(4, 136), k=pages(2, 136),
                v=pages(2, 136)) == EUNSUP
    assert call(B=1 << 30, ts=0) == EUNSUP
    for name in ("k", "v"):
        assert call(**{name: pages(p=None)}) == EINVAL
        assert call(**{name: pages(p=FAKE + 8)}) == EALIGN
        assert call(**{name: pages(token=132)}) == EALIGN
        assert call(**{name: pages(page=8)}) == EINVAL
    assert call(q=rows(4, p=None)) == EINVAL and call(out=rows(4, head=3)) == EINVAL
    assert call(ws=None) == EWS and call(wsn=need - 1) == EWS and call(ws=FAKE + 128) == EWS


def test_append_errors(lib):
    def call(**kw):
        a = dict(q=rows(4), k=rows(), v=rows(), T=10, hq=4, hkv=2, d=64, dt=0, kc=pages(),
                 vc=pages(), n=9, size=16, table=FAKE, ts=5, mp=5, start=FAKE, cu=FAKE, B=2,
                 pos=None, ps=0, inv=FAKE, pairs=32, axes=1, paired=0, qo=rows(4),
                 ko=_lib.Rows(None, 0, 0))
        a.update(kw)
        return lib.rnn_kv_append(ctypes.byref(_lib.KvAppendArgs(
            q=a["q"], k=a["k"], v=a["v"], q_out=a["qo"], k_out=a["ko"], k_cache=a["kc"],
            v_cache=a["vc"], page_table=a["table"], start=a["start"], cu=a["cu"],
            positions=a["pos"], inv_freq=a["inv"], T=a["T"], num_pages=a["n"],
            table_stride=a["ts"], position_stride=a["ps"], Hq=a["hq"], Hkv=a["hkv"], d=a["d"],
            dtype=a["dt"], page_size=a["size"], max_pages=a["mp"], B=a["B"], pairs=a["pairs"],
            axes=a["axes"], paired=a["paired"])), None)

    assert lib.rnn_kv_append(None, None) == EINVAL

    assert call(T=-1) == EINVAL and call(B=-1) == EINVAL and call(hkv=0) == EINVAL
    assert call(d=20) == EALIGN and call(dt=2) == EINVAL and call(mp=0) == EINVAL
    assert call(d=264, pairs=0, axes=0) == EUNSUP
    assert call(pairs=33) == EINVAL and call(pairs=0) == EINVAL and call(axes=0) == EINVAL
    assert call(axes=3, pairs=8) == EINVAL and call(inv=None) == EINVAL
    assert call(inv=FAKE + 4) == EINVAL
    assert call(axes=2, pairs=16) == EINVAL                       # two axes need positions
    assert call(axes=2, pairs=16, pos=FAKE, ps=1) == EINVAL       # rows of positions overlap
    assert call(start=None) == EINVAL and call(cu=FAKE + 1) == EINVAL and call(table=None) == EINVAL
    for name, h in (("q", 4), ("k", 2), ("v", 2), ("qo", 4), ("ko", 2)):
        assert call(**{name: rows(h, p=FAKE + 2)}) == EALIGN
        assert call(**{name: rows(h, token=8)}) == EINVAL
    for name in ("kc", "vc"):
        assert call(**{name: pages(head=70)}) == EALIGN
        assert call(**{name: pages(p=None)}) == EINVAL


def test_binding_refuses_cpu_tensors():
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    c = torch.zeros((2, 16, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        rnn.attn_prompt(x, x, x, i)
    with pytest.raises(ValueError):
        rnn.attn_decode(x, c, c, torch.zeros((4, 2), dtype=torch.int32), i)
    with pytest.raises(ValueError):
        rnn.kv_append(x, x, c, c, torch.zeros((1, 2), dtype=torch.int32), i[:1], i)
    with pytest.raises(TypeError):
        rnn.attn_prompt(x.float(), x, x, i)


class OnGpu:
    """A stand-in for a CUDA tensor, enough for the checks before the first launch."""

    def __new__(cls, *shape, dtype=torch.bfloat16, strides=None, device="cuda:0"):
        t = torch.empty(shape, dtype=dtype)
        if strides is not None:
            t = torch.empty(1 << 16, dtype=dtype).as_strided(shape, strides)
        return t.as_subclass(_Fake)


class _Fake(torch.Tensor):
    @property
    def is_cuda(self):
        return True

    @property
    def device(self):
        return torch.device("cpu")


def test_binding_checks_shapes_types_and_strides():
    I = dict(dtype=torch.int32)
    q, k = OnGpu(8, 4, 64), OnGpu(8, 2, 64)
    cu = OnGpu(3, **I)
    bad = [
        (TypeError, (q.half(), k, k, cu), {}),
        (ValueError, (q, OnGpu(8, 3, 64), OnGpu(8, 3, 64), cu), {}),
        (ValueError, (q, k, OnGpu(9, 2, 64), cu), {}),
        (ValueError, (q, OnGpu(8, 2, 32), OnGpu(8, 2, 32), cu), {}),
        (ValueError, (OnGpu(8, 4, 136), OnGpu(8, 2, 136), OnGpu(8, 2, 136), cu), {}),
        (TypeError, (q, k, k, OnGpu(3, dtype=torch.int64)), {}),
        (ValueError, (q, k, k, OnGpu(0, **I)), {}),
        (ValueError, (q, k, k, cu, OnGpu(4, **I)), {}),
        (ValueError, (q, k, k, OnGpu(3, dtype=torch.int32, strides=(2,))), {}),
        (ValueError, (q, k, k, cu), dict(scale=-1.0)),
        (ValueError, (q, k, k, cu), dict(scale=float("inf"))),
        (ValueError, (q, k, k, cu), dict(out=OnGpu(8, 2, 64))),
        (ValueError, (OnGpu(8, 4, 64, strides=(256, 64, 2)), k, k, cu), {}),
        (ValueError, (OnGpu(8, 4, 64, strides=(260, 64, 1)), k, k, cu), {}),
        (ValueError, (q, OnGpu(8, 2, 64, strides=(64, 0, 1)), k, cu), {}),
    ]
    for err, args, kw in bad:
        with pytest.raises(err):
            rnn.attn_prompt(*args, **kw)
    c = OnGpu(5, 16, 2, 64)
    tab, lens = OnGpu(8, 3, **I), OnGpu(8, **I)
    bad = [
        (ValueError, (q, c, OnGpu(5, 8, 2, 64), tab, lens)),
        (ValueError, (q, OnGpu(5, 16, 2, 32), OnGpu(5, 16, 2, 32), tab, lens)),
        (ValueError, (q, c, c, OnGpu(7, 3, **I), lens)),
        (ValueError, (q, c, c, OnGpu(8, 0, **I), lens)),
        (TypeError, (q, c, c, tab, OnGpu(8, dtype=torch.int64))),
        (ValueError, (q, c, c, tab, OnGpu(9, **I))),
        (TypeError, (q, c.half(), c.half(), tab, lens)),
        (ValueError, (q, OnGpu(0, 16, 2, 64), OnGpu(0, 16, 2, 64), tab, lens)),
    ]
    for err, args in bad:
        with pytest.raises(err):
            rnn.attn_decode(*args)
    tab, start = OnGpu(2, 3, **I), OnGpu(2, **I)
    inv = OnGpu(32, dtype=torch.float64)
    ok = (k, k, c, c, tab, start, cu)
    bad = [
        (ValueError, ok, dict(q=q)),                                      # nothing to rotate by
        (ValueError, ok, dict(q_out=q)),
        (ValueError, ok, dict(inv_freq=OnGpu(33, dtype=torch.float64))),  # 66 channels of 64
        (TypeError, ok, dict(inv_freq=OnGpu(32, dtype=torch.float32))),
        (ValueError, ok, dict(inv_freq=OnGpu(0, dtype=torch.float64))),
        (ValueError, ok, dict(positions=OnGpu(8, **I))),                  # positions alone
        (ValueError, ok, dict(inv_freq=inv, positions=OnGpu(7, **I))),
        (ValueError, ok, dict(inv_freq=inv, positions=OnGpu(8, 2, **I))),  # 128 channels of 64
        (ValueError, ok, dict(inv_freq=inv, positions=OnGpu(8, 3, **I))),
        (ValueError, ok, dict(inv_freq=inv, q=OnGpu(7, 4, 64))),
        (ValueError, ok, dict(k_out=OnGpu(8, 4, 64))),
        (ValueError, (k, k, c, c, tab, OnGpu(3, **I), cu), {}),
        (ValueError, (k, OnGpu(8, 4, 64), c, c, tab, start, cu), {}),
        (ValueError, (OnGpu(8, 2, 264), OnGpu(8, 2, 264), OnGpu(5, 16, 2, 264),
                      OnGpu(5, 16, 2, 264), tab, start, cu), {}),
    ]
    for err, args, kw in bad:
        with pytest.raises(err):
            rnn.kv_append(*args, **kw)
