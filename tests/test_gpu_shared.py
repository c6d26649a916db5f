"""Attention behind a shared prefix against the double-precision oracle (needs a B200)."""
import math

import numpy as np
import pytest
import torch

import reciprocal_nearest_neighbour_b200 as rnn
from attn_bounds import check_attention
from oracle import attention as oa
from oracle.shared import decode_shared

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def f64(t):
    return t.double().cpu().numpy()


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def gen_of(seed):
    return torch.Generator().manual_seed(seed)


def normal(gen, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=gen, dtype=torch.float32) * std).to(dtype).cuda()


def setting(dtype, prefix, lens, hq, hkv, d, size, seed=0, std=1.0, layout="plain"):
    g = gen_of(seed)
    need = [-(-n // size) for n in lens]
    pre = max(1, -(-prefix // size))
    pages = sum(need) + pre + 2
    order = torch.randperm(pages, generator=g).tolist()
    table = np.full((len(lens), max(need + [1])), -1, dtype=np.int64)
    for b, n in enumerate(need):
        table[b, :n] = [order.pop() for _ in range(n)]
    names = np.array([order.pop() for _ in range(pre)])

    def cache():
        if layout == "head":
            return normal(g, (pages, hkv, size, d), dtype, std).transpose(1, 2)
        if layout == "wide":
            return normal(g, (pages, size, hkv, d + 24), dtype, std)[..., 16:16 + d]
        return normal(g, (pages, size, hkv, d), dtype, std)

    kc, vc = cache(), cache()
    q = normal(g, (len(lens), hq + 3, d + 8), dtype, std)[:, 2:2 + hq, 8:] if layout == "wide" else \
        normal(g, (len(lens), hq, d), dtype, std)
    return q, kc, vc, names, table


def run_shared(dtype, prefix, lens, hq, hkv, d, size, scale=None, change=None, **kw):
    q, kc, vc, names, table = setting(dtype, prefix, lens, hq, hkv, d, size, **kw)
    if change:
        change(q, kc, vc, names, table)
    ws = torch.full((rnn.attn._shared_need(len(lens), hq, hkv, d, len(names) * size),), 255,
                    dtype=torch.uint8, device="cuda")    # NaN wherever it is read unwritten
    out = torch.full_like(q, 7.0, memory_format=torch.contiguous_format)
    got, lse = rnn.attn_decode_shared(q, kc, vc, ints(names), ints([prefix]), ints(table), ints(lens),
                                      scale=scale, with_lse=True, out=out, workspace=ws)
    assert got is out
    rnn.workspace_status(ws)
    ref = decode_shared(f64(q), f64(kc), f64(vc), names, prefix, table, lens,
                        1 / math.sqrt(d) if scale is None else scale)
    check_attention(out, lse, ref, dtype, d, float(vc.abs().max()))
    return q, kc, vc, names, table, out, lse


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d", [8, 24, 40, 64, 72, 96, 112, 128])
def test_depths(dtype, d):
    run_shared(dtype, 300, [5, 70, 1], 4, 2, d, 16, seed=d)


@pytest.mark.parametrize("prefix", [1, 2, 127, 128, 129, 255, 256, 257, 600, 2000])
@pytest.mark.parametrize("d", [64, 128])
def test_prefix_lengths(prefix, d):
    run_shared(HF, prefix, [3, 1, 40], 2, 1, d, 16, seed=prefix)


@pytest.mark.parametrize("batch,hq,hkv", [(1, 1, 1), (2, 7, 1), (16, 8, 1), (43, 3, 1), (64, 4, 2),
                                          (65, 2, 1), (128, 2, 2), (129, 2, 1), (200, 2, 1),
                                          (33, 40, 2), (400, 1, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_rows(batch, hq, hkv, d):
    """Rows of a key head: one to several units, the last of them wide or narrow, full or not."""
    rng = np.random.default_rng(batch)
    run_shared(BF, 700, rng.integers(0, 20, batch).tolist(), hq, hkv, d, 16, seed=batch)


@pytest.mark.parametrize("size", [1, 3, 8, 16, 24, 48, 100, 128, 256])
@pytest.mark.parametrize("layout", ["plain", "head", "wide"])
def test_pages(size, layout):
    run_shared(HF, 413, [0, 1, 31, 33, 130], 4, 2, 64, size, seed=size, layout=layout)
    run_shared(BF, 260, [9, 0], 6, 2, 96, size, seed=size, layout=layout)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_empty_parts(dtype):
    run_shared(dtype, 0, [3, 0, 500], 4, 2, 64, 16)       # no prefix, and a row without a key
    run_shared(dtype, 333, [0, 0, 0], 4, 2, 128, 16)      # nothing of their own
    run_shared(dtype, 0, [0, 0], 2, 2, 64, 16)
    run_shared(dtype, -5, [2, -3], 2, 1, 64, 16)


@pytest.mark.parametrize("d", [64, 128])
def test_pages_that_do_not_exist(d):
    def some(q, kc, vc, names, table):
        names[1], names[3], names[-1], table[0, 0] = -1, 99999, -7, -1

    def every(q, kc, vc, names, table):
        names[:] = -1

    run_shared(BF, 700, [20, 3], 4, 2, d, 16, change=some)
    run_shared(BF, 700, [20, 3], 4, 2, d, 128, change=some)
    run_shared(HF, 700, [20, 0], 4, 2, d, 24, change=every)


def test_lengths_beyond_the_tables():
    q, kc, vc, names, table = setting(HF, 40, [5, 30], 2, 1, 64, 16)
    args = (q, kc, vc, ints(names))
    got = rnn.attn_decode_shared(*args, ints([10 ** 9]), ints(table), ints([2 ** 31 - 1, 32]))
    want = rnn.attn_decode_shared(*args, ints([48]), ints(table), ints([32, 32]))
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("batch", [3, 70])
def test_growing_scores(dtype, d, batch):
    """Every key tile's scores exceed the last one's, so every tile rescales."""
    def change(q, kc, vc, names, table):
        size = kc.shape[1]
        n = len(names) * size
        ramp = torch.linspace(-8, 8, n, device="cuda").to(dtype)
        kc.mul_(0.1)
        for j, page in enumerate(names):
            kc[page] += ramp[j * size:(j + 1) * size, None, None]
        q.mul_(0.5).add_(1.0)

    run_shared(dtype, 1400, [4] * batch, 4, 1, d, 16, change=change)


@pytest.mark.parametrize("scale,std", [(40.0, 1.0), (1e-30, 1.0), (3e7, 1.0), (None, 1e-3)])
def test_scores_of_any_size(scale, std):
    def sharp(q, kc, vc, names, table):
        # scores that are whole numbers, so that the largest scale keeps them exact
        for t in (q, kc):
            t.copy_(t.float().round().clamp(-2, 2).to(t.dtype))

    run_shared(BF, 300, [5, 40, 0], 2, 1, 64, 16, scale=scale, std=std,
               change=sharp if scale == 3e7 else None)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_is_not_finite_shows(dtype, d, bad):
    """In the prefix every row of the head is NaN, in a sequence's own keys its rows are."""
    q, kc, vc, names, table = setting(dtype, 300, [20, 33], 4, 2, d, 16, seed=3)
    q[:, :, 0] = 1.0
    args = (ints(names), ints([300]), ints(table), ints([20, 33]))
    good, good_lse = rnn.attn_decode_shared(q, kc, vc, *args, with_lse=True)
    kept = kc[table[1, 1], 2, 0, 0].clone()
    kc[table[1, 1], 2, 0, 0] = bad
    out, lse = rnn.attn_decode_shared(q, kc, vc, *args, with_lse=True)
    assert torch.equal(out[0], good[0]) and torch.equal(out[1, 2:], good[1, 2:])
    assert out[1, :2].isnan().all() and lse[1, :2].isnan().all()
    kc[table[1, 1], 2, 0, 0] = kept
    kc[names[5], 3, 1, 0] = bad
    out, lse = rnn.attn_decode_shared(q, kc, vc, *args, with_lse=True)
    assert torch.equal(out[:, :2], good[:, :2]) and torch.equal(lse[:, :2], good_lse[:, :2])
    assert out[:, 2:].isnan().all() and lse[:, 2:].isnan().all()
    kc[names, :, 1, 0] = float("nan")                     # a head without a single number
    kc[table[0], :, 1, 0] = float("nan")
    out, lse = rnn.attn_decode_shared(q, kc, vc, *args, with_lse=True)
    assert out[0, 2:].isnan().all() and lse[0, 2:].isnan().all()


def test_rows_behind_the_last_key_may_hold_anything():
    q, kc, vc, names, table = setting(HF, 131, [20, 33], 4, 2, 64, 16, seed=3)
    args = (ints(names), ints([131]), ints(table), ints([20, 33]))
    want = rnn.attn_decode_shared(q, kc, vc, *args)
    for t in (kc, vc):
        t[names[-1], 131 % 16:] = float("nan")
        t[table[0, 1], 4:] = float("inf")
    assert torch.equal(rnn.attn_decode_shared(q, kc, vc, *args), want)


@pytest.mark.parametrize("batch,d", [(6, 64), (150, 128)])
def test_the_same_bits_again(batch, d):
    q, kc, vc, names, table = setting(BF, 5000, [40] * batch, 4, 1, d, 16)
    args = (q, kc, vc, ints(names), ints([5000]), ints(table), ints([40] * batch))
    a, b = (rnn.attn_decode_shared(*args) for _ in range(2))
    assert torch.equal(a, b)


def test_as_one_long_sequence():
    """The prefix and a tail give what attn_decode gives for the sequence they make."""
    B, hq, hkv, d, size, prefix = 5, 8, 2, 128, 16, 640
    g = gen_of(8)
    lens = [1, 16, 3, 100, 40]
    inv = (10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)).cuda()
    # the prefix's tokens, once
    pages = prefix // size + B * 8
    kc, vc = (torch.zeros(pages, size, hkv, d, dtype=HF, device="cuda") for _ in range(2))
    names = ints(range(prefix // size))
    k, v = (normal(g, (prefix, hkv, d), HF) for _ in range(2))
    rnn.kv_append(k, v, kc, vc, names[None], ints([0]), ints([0, prefix]), inv_freq=inv)
    # each sequence's own, numbered behind it
    table = prefix // size + torch.arange(B * 8, dtype=torch.int32, device="cuda").view(B, 8)
    cu = [0] + np.cumsum(lens).tolist()
    k, v = (normal(g, (cu[-1], hkv, d), HF) for _ in range(2))
    at = ints(np.concatenate([prefix + np.arange(n) for n in lens]))
    rnn.kv_append(k, v, kc, vc, table, ints([0] * B), ints(cu), inv_freq=inv, positions=at)
    q = normal(g, (B, hq, d), HF)
    got, got_lse = rnn.attn_decode_shared(q, kc, vc, names, ints([prefix]), table, ints(lens), with_lse=True)
    long = torch.cat([names[None].expand(B, -1), table], 1).contiguous()
    want, want_lse = rnn.attn_decode(q, kc, vc, long, ints([prefix + n for n in lens]), with_lse=True)
    ref = oa.decode(f64(q), f64(kc), f64(vc), f64(long).astype(int), [prefix + n for n in lens], d ** -0.5)
    for out, lse in ((got, got_lse), (want, want_lse)):
        check_attention(out, lse, ref, HF, d, float(vc.abs().max()))


def test_graph_streams_and_shared_workspaces():
    """Captured twice on one workspace, replayed with other lengths and inputs; another stream."""
    lens = [20, 33, 7]
    q, kc, vc, names, table = setting(BF, 500, lens, 4, 2, 128, 16, seed=5)
    pre_len, own, tab, nam = ints([500]), ints(lens), ints(table), ints(names)
    ws = torch.empty(rnn.attn._shared_need(3, 4, 2, 128, len(names) * 16), dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(q) for _ in range(2)]

    def step(i):
        rnn.attn_decode_shared(q, kc, vc, nam, pre_len, tab, own, out=outs[i], workspace=ws,
                               scale=0.05 * (i + 1))

    step(0)
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(i)
        graphs.append(graph)
    for prefix, mine in ((500, lens), (130, [1, 0, 33]), (0, [5, 5, 5])):
        pre_len.fill_(prefix)
        own.copy_(ints(mine))
        q.copy_(normal(gen_of(prefix), tuple(q.shape), BF))
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        rnn.workspace_status(ws)
        got = [o.clone() for o in outs]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            fresh = [rnn.attn_decode_shared(q, kc, vc, nam, pre_len, tab, own, scale=0.05 * (i + 1))
                     for i in range(2)]
        side.synchronize()
        for a, b in zip(got, fresh):
            assert torch.equal(a, b)


@pytest.mark.parametrize("d,batch", [(64, 3), (128, 3), (128, 150)])
def test_wait_runs_out_and_is_reported(d, batch):
    """Loads that never come: rows NaN, the status word set, and the next call is whole."""
    q, kc, vc, names, table = setting(HF, 300, [20] * batch, 2, 1, d, 16)
    args = (q, kc, vc, ints(names), ints([300]), ints(table), ints([20] * batch))
    ws = torch.empty(rnn.attn._shared_need(batch, 2, 1, d, len(names) * 16), dtype=torch.uint8, device="cuda")
    want = rnn.attn_decode_shared(*args)
    lib = rnn._lib.load()
    lib.rnn_test_stall_loads(1, 2_000_000)
    try:
        out, lse = rnn.attn_decode_shared(*args, workspace=ws, with_lse=True)
        torch.cuda.synchronize()
    finally:
        lib.rnn_test_stall_loads(0, 0)
    with pytest.raises(rnn.RNNError) as e:
        rnn.workspace_status(ws)
    assert e.value.name == "RNN_ETIMEOUT"
    assert out.isnan().all() and lse.isnan().all()
    again = rnn.attn_decode_shared(*args, workspace=ws)
    rnn.workspace_status(ws)
    assert torch.equal(again, want)


@pytest.mark.parametrize("batch", [0, 3])
def test_the_word_is_cleared(batch):
    q = torch.ones((batch, 2, 64), dtype=HF, device="cuda")
    cache = torch.ones((2, 16, 1, 64), dtype=HF, device="cuda")
    need = rnn.attn._shared_need(batch, 2, 1, 64, 16)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    out = rnn.attn_decode_shared(q, cache, cache, ints([0]), ints([9]), ints(np.ones((batch, 1))),
                                 ints([20] * batch), workspace=ws)
    rnn.workspace_status(ws)
    assert (out == 1).all()


def test_a_long_prefix():
    """More keys than one accumulator takes: 300 000 of one sign."""
    g = gen_of(2)
    n, size, d = 300000, 256, 64
    pages = -(-n // size)
    kc, vc = (normal(g, (pages + 1, size, 1, d), HF, 0.5) for _ in range(2))
    vc.abs_()
    q = normal(g, (2, 2, d), HF)
    names = np.arange(pages)
    out, lse = rnn.attn_decode_shared(q, kc, vc, ints(names), ints([n]), ints([[pages], [pages]]),
                                      ints([1, 9]), with_lse=True)
    ref = decode_shared(f64(q), f64(kc), f64(vc), names, n, np.array([[pages], [pages]]), [1, 9], 1 / 8)
    # each sum leaves its accumulator after 65536 keys at most: 2^-11 of it may be cut off
    ref.spread *= 1 + 2.0 ** -11 / 2.0 ** -11
    check_attention(out, lse, ref, HF, d, float(vc.max()))


def test_python_form_gives_the_same(monkeypatch):
    """The call's way through the extension module and the one through Python."""
    q, kc, vc, names, table = setting(BF, 300, [20, 3], 4, 2, 64, 16)
    args = (q, kc, vc, ints(names), ints([300]), ints(table), ints([20, 3]))
    mine = rnn.attn_decode_shared(*args, with_lse=True, scale=0.2)
    monkeypatch.setattr(rnn._lib, "fast", rnn._lib._Python)
    for x, y in zip(mine, rnn.attn_decode_shared(*args, with_lse=True, scale=0.2)):
        assert torch.equal(x, y)


def test_more_rows_than_a_wave():
    rng = np.random.default_rng(0)
    run_shared(BF, 150, rng.integers(0, 4, 3000).tolist(), 2, 2, 32, 16)


def test_pages_may_repeat():
    def change(q, kc, vc, names, table):
        names[2], names[4], table[1] = names[0], names[0], table[0]

    run_shared(HF, 200, [30, 30], 4, 2, 64, 16, change=change)


@pytest.mark.parametrize("d", [64, 128])
def test_offsets_beyond_32_bits(d):
    """Pages 1.3 10^9 elements apart."""
    g = gen_of(1)
    size, hkv, gap = 16, 2, 1300000000 // 8 * 8
    store = torch.empty(3 * gap, dtype=HF, device="cuda")
    shape, strides = (4, size, hkv, d), (gap // 2 // 8 * 8, hkv * d, d, 1)
    kc = store.as_strided(shape, strides)
    vc = store[gap // 4 // 8 * 8:].as_strided(shape, strides)
    for c in (kc, vc):
        c.copy_(normal(g, shape, HF))
    q = normal(g, (2, 4, d), HF)
    names, table, lens = np.array([3, 0]), np.array([[2], [1]]), [16, 5]
    out, lse = rnn.attn_decode_shared(q, kc, vc, ints(names), ints([30]), ints(table), ints(lens), with_lse=True)
    ref = decode_shared(f64(q), f64(kc), f64(vc), names, 30, table, lens, d ** -0.5)
    check_attention(out, lse, ref, HF, d, float(vc.abs().max()))


def test_two_calls_at_once():
    """Two streams, a workspace each, and a prompt beside them."""
    sets = [setting(BF, 2000, [40] * 60, 4, 1, 128, 16, seed=s) for s in (1, 2)]
    args = [(q, kc, vc, ints(names), ints([2000]), ints(table), ints([40] * 60)) for q, kc, vc, names, table in sets]
    want = [rnn.attn_decode_shared(*a) for a in args]
    x = normal(gen_of(3), (1500, 4, 128), BF)
    cu = ints([0, 1500])
    whole = rnn.attn_prompt(x, x, x, cu)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [[], [], []]
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(rnn.attn_decode_shared(*args[i]))
        with torch.cuda.stream(streams[2]):
            got[2].append(rnn.attn_prompt(x, x, x, cu))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])
    assert all(torch.equal(y, whole) for y in got[2])
