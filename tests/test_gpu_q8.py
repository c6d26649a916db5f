"""The cache in 8-bit codes against the double-precision oracle (needs a B200)."""
import math

import numpy as np
import pytest
import torch

import reciprocal_nearest_neighbour_b200 as rnn
from oracle import attention as oa
from oracle import cache_q8 as oq
from q8_bounds import check_attention_q8, turn_error

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
CODES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def f64(t):
    return t.double().cpu().numpy()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cum(lens):
    return [0] + np.cumsum(lens).tolist()


def gen_of(seed):
    return torch.Generator().manual_seed(seed)


def normal(gen, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=gen, dtype=torch.float32) * std).to(dtype).cuda()


def raw(t):
    return t.view(torch.uint8).cpu().numpy()


def strided(pages, size, heads, d, layout):
    """A byte cache in one of several orders, filled with 0x5A."""
    if layout == "head":        # heads outermost in a page
        return torch.full((pages, heads, size, d), 0x5A, dtype=torch.uint8,
                          device="cuda").transpose(1, 2)
    if layout == "wide":        # rows 8 bytes wider than they need to be, 8 bytes in
        t = torch.full((pages, size, heads, d + 24), 0x5A, dtype=torch.uint8, device="cuda")
        return t[..., 16:16 + d]
    return torch.full((pages, size, heads, d), 0x5A, dtype=torch.uint8, device="cuda")


def new_cache(codes, pages, size, heads, d, layout="plain"):
    kc, vc = (strided(pages, size, heads, d, layout).view(CODES[codes]) for _ in range(2))
    scales = torch.full((pages, heads, size, 2), 7.0, device="cuda")
    if layout == "wide":        # a slice of more heads and rows
        scales = torch.full((pages, heads + 1, size + 3, 2), 7.0, device="cuda")[:, 1:, :size]
    return kc, vc, scales


def filled(gen, codes, pages, size, heads, d, layout="plain", spread=0.5):
    """A cache as an append would leave it, and the values that it stands for."""
    kc, vc, scales = new_cache(codes, pages, size, heads, d, layout)
    values = []
    for which, cache in enumerate((kc, vc)):
        x = torch.randn(pages, size, heads, d, generator=gen)
        x *= torch.exp(spread * torch.randn(pages, size, heads, 1, generator=gen))
        v, s = oq.quantise32(x.numpy(), codes)
        cache.copy_(torch.from_numpy(v).to(CODES[codes]).cuda()) if codes == "int8" else \
            cache.view(torch.uint8).copy_(torch.from_numpy(v).to(CODES[codes]).view(torch.uint8).cuda())
        scales[..., which] = torch.from_numpy(s).transpose(1, 2).cuda()
        values.append(v * s[..., None].astype(np.float64))
    return kc, vc, scales, values[0], values[1]


def deal(gen, totals, size, extra=2):
    """Pages of the sequences in a random order, and their number."""
    need = [-(-n // size) for n in totals]
    order = torch.randperm(sum(need) + extra, generator=gen).tolist()
    table = np.full((len(totals), max(need + [1])), -1, dtype=np.int64)
    for b, n in enumerate(need):
        table[b, :n] = [order.pop() for _ in range(n)]
    return table, sum(need) + extra


# ------------------------------------------------------------------ append
def run_append(codes, dtype, new, past, hq, hkv, d, size, pairs=0, axes=1, paired=False,
               layout="plain", seed=0, with_k=False, in_place=False, front=0, behind=0):
    g = gen_of(seed)
    T = front + sum(new) + behind
    rows = normal(g, (T, hq + 2 * hkv, d), dtype)
    q, k, v = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]
    totals = [a + b for a, b in zip(new, past)]
    table, pages = deal(g, totals, size)
    kc, vc, scales = new_cache(codes, pages, size, hkv, d, layout)
    before = [raw(kc).copy(), raw(vc).copy()]
    cu = [front + c for c in cum(new)]
    inv = None if not pairs else 10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)
    pos = None
    if axes == 2:
        pos = torch.randint(0, 500, (T, 2), generator=g, dtype=torch.int32)
    q0, k0 = f64(q), f64(k)
    kw = {}
    if pairs and hq:
        kw["q"] = q
    if in_place:
        kw.update(q_out=q, k_out=k)
    out, k_out = rnn.kv_append_q8(
        k, v, kc, vc, scales, ints(table), ints(past), ints(cu),
        inv_freq=None if inv is None else inv.cuda(), positions=None if pos is None else pos.cuda(),
        paired=paired, with_k=with_k, **kw)
    where, number = oa.slots(cu, past, table, size, pages, T)
    u = torch.finfo(dtype).eps / 2
    want_k, want_q = k0.copy(), q0.copy()
    inside = slice(front, T - behind)
    if pairs:
        at = np.array([[0 if n is None else n] for n in number]) if pos is None else pos.numpy()
        want_k, want_q = (oa.rotate(x, at, inv.numpy(), paired) for x in (k0, q0))

    def reach(x):               # |x1| + |x2| of a channel's pair, 0 where nothing turns
        r = np.zeros_like(x)
        for a in range(axes if pairs else 0):
            for i in range(pairs):
                one = 2 * pairs * a + (2 * i if paired else i)
                two = one + (1 if paired else pairs)
                r[..., one] = r[..., two] = np.abs(x[..., one]) + np.abs(x[..., two])
        return r

    if "q" in kw:
        tol = u * np.abs(want_q) + turn_error * reach(q0) * 1.01 + 2.0 ** -25
        assert np.all(np.abs(f64(out) - want_q)[inside] <= tol[inside])
    else:
        assert out is None
    if with_k or in_place:
        tol = u * np.abs(want_k) + turn_error * reach(k0) * 1.01 + 2.0 ** -25
        assert np.all(np.abs(f64(k_out) - want_k)[inside] <= tol[inside])
    else:
        assert k_out is None
    got = [raw(kc), raw(vc)]
    sc = scales.cpu().numpy()
    touched = np.zeros(got[0].shape[:2], dtype=bool)
    v32 = v.float().cpu().numpy()
    for t in range(T):
        if where[t] is None:
            continue
        pg, row = where[t]
        touched[pg, row] = True
        # values: fp32's own quotients, to the bit
        cv, s = oq.quantise32(v32[t], codes)
        assert np.array_equal(sc[pg, :, row, 1], s)
        assert np.array_equal(oq.value(got[1][pg, row], codes), cv)
        slack = turn_error * 1.01 * reach(k0[t])
        if not pairs:
            ck, s = oq.quantise32(k0[t], codes)
            assert np.array_equal(sc[pg, :, row, 0], s)
            assert np.array_equal(oq.value(got[0][pg, row], codes), ck)
            continue
        s = sc[pg, :, row, 0].astype(np.float64)
        want = oq.scale(want_k[t], codes)
        assert np.all(np.abs(s - want) <= 2.0 ** -23 * want + slack.max(-1) / oq.TOP[codes])
        held = oq.value(got[0][pg, row], codes) * s[:, None]
        far = (np.abs(want_k[t]) + slack) / s[:, None]
        tol = oq.half_step(far, codes) * s[:, None] + slack + 3 * 2.0 ** -23 * np.abs(want_k[t])
        assert np.all(np.abs(held - want_k[t]) <= tol)
    for a, b in zip(got, before):
        assert np.array_equal(a[~touched], b[~touched])
    keep = np.broadcast_to(~touched[:, None, :, None], sc.shape)
    assert np.all(sc[keep] == 7.0)
    return kc, vc, scales, table, cu


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d", [8, 24, 40, 64, 72, 128, 136, 256])
def test_append_depths(codes, dtype, d):
    run_append(codes, dtype, [5, 0, 17], [3, 9, 0], 4, 2, d, 16, pairs=d // 2, seed=d)


@pytest.mark.parametrize("paired", [False, True])
@pytest.mark.parametrize("pairs,axes", [(32, 1), (16, 1), (16, 2), (12, 1), (10, 2), (5, 1), (3, 2), (1, 1)])
def test_append_rotations(pairs, axes, paired):
    run_append("e4m3", BF, [9, 30], [700, 0], 3, 1, 64, 16, pairs, axes, paired, seed=pairs)
    run_append("int8", HF, [9, 30], [700, 0], 3, 3, 72, 24, pairs, axes, paired, seed=pairs)


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
@pytest.mark.parametrize("layout", ["plain", "head", "wide"])
@pytest.mark.parametrize("size", [1, 7, 16, 100])
def test_append_caches(codes, layout, size):
    run_append(codes, HF, [1, 40, 2], [0, 5, 33], 6, 3, 40, size, pairs=20, layout=layout,
               seed=size, front=2, behind=3)


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
def test_append_without_rotation(codes):
    run_append(codes, BF, [33], [2], 0, 5, 96, 8)
    run_append(codes, HF, [1], [0], 0, 1, 64, 16)


@pytest.mark.parametrize("d,pairs,paired", [(64, 32, False), (128, 64, False), (72, 20, False), (64, 16, True)])
def test_append_in_place(d, pairs, paired):
    run_append("int8", HF, [40, 3], [1, 2], 4, 2, d, 16, pairs=pairs, paired=paired, in_place=True)
    run_append("e4m3", BF, [300], [1], 2, 2, d, 16, pairs=pairs, paired=paired, with_k=True)


def test_append_many_tokens():
    run_append("e4m3", BF, [2600, 500], [0, 77], 1, 1, 32, 64, pairs=16, seed=3)


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
def test_append_sizes_of_values(codes):
    """Zeros, subnormals, the type's largest, and rows that hold what is not finite."""
    d = 64
    x = torch.zeros(8, 1, d, dtype=BF)
    x[1] = 1e-40
    x[2, 0, 3] = 3e38
    x[3] = torch.linspace(-1, 1, d)
    x[4, 0, 5] = float("nan")
    x[5, 0, 5] = float("inf")
    x[6, 0, 5], x[6, 0, 6] = float("-inf"), float("nan")
    x[7] = 2.0 ** -126
    x = x.cuda()
    kc, vc, scales = new_cache(codes, 1, 8, 1, d)
    args = (kc, vc, scales, ints([[0]]), ints([0, 8]))
    rnn.kv_append_q8(x, x, kc, vc, scales, ints([[0]]), ints([0]), ints([0, 8]))
    k, v = rnn.kv_read_q8(*args, 8, BF)
    assert torch.equal(k.view(torch.int16), v.view(torch.int16))
    good = [0, 1, 2, 3, 7]
    cv, s = oq.quantise32(x[good].float().cpu().numpy(), codes)
    assert np.array_equal(scales[0, 0, good, 0].cpu().numpy(), s[:, 0])
    assert np.array_equal(oq.value(raw(kc)[0, good], codes), cv)
    assert scales[0, 0, 4:7].isnan().all() and k[4:7].isnan().all()
    assert k[good].isfinite().all()


def test_append_tokens_that_do_not_exist():
    """Numbers outside the table and pages outside the cache: rotated, not stored."""
    d, size = 64, 4
    x = normal(gen_of(1), (12, 1, d), HF)
    kc, vc, scales = new_cache("e4m3", 3, size, 1, d)
    inv = torch.ones(8, dtype=torch.float64, device="cuda")
    table = ints([[2, -1, 7]])
    q, k = rnn.kv_append_q8(x, x, kc, vc, scales, table, ints([-2]), ints([0, 12]), q=x,
                            inv_freq=inv, with_k=True)
    at = np.arange(-2, 10)[:, None]
    want = oa.rotate(f64(x), at, np.ones(8), False)
    assert np.abs(f64(q) - want).max() < 4e-3 and torch.equal(q, k)
    assert (raw(kc)[[0, 1]] == 0x5A).all() and (raw(vc)[[0, 1]] == 0x5A).all()
    assert not (raw(vc)[2] == 0x5A).all(-1).any() and (scales[:2] == 7).all()


# -------------------------------------------------------------------- read
@pytest.mark.parametrize("codes", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d,size,layout", [(8, 1, "plain"), (40, 7, "plain"), (64, 16, "head"), (72, 24, "wide"), (128, 16, "plain"), (256, 5, "plain")])
def test_read(codes, dtype, d, size, layout):
    g = gen_of(d)
    lens, hkv, front = [0, 5, 61, 1, 0, 200], 3, 2
    first = [0, 2, 0, 9, 4, 0]
    table, pages = deal(g, [a + b for a, b in zip(lens, first)], size)
    kc, vc, scales, _, _ = filled(g, codes, pages, size, hkv, d, layout)
    table[2, 0], table[5, -1] = -1, pages                   # two pages that do not exist
    cu = [front + c for c in cum(lens)]
    T = cu[-1] + 4
    outs = [torch.full((T, hkv, d), 3.0, dtype=dtype, device="cuda") for _ in range(2)]
    got = rnn.kv_read_q8(kc, vc, scales, ints(table), ints(cu), T, dtype, start=ints(first),
                         k_out=outs[0], v_out=outs[1])
    assert got[0] is outs[0] and got[1] is outs[1]
    where, _ = oa.slots(cu, first, table, size, pages, T)
    for which, (cache, out) in enumerate(zip((kc, vc), outs)):
        codes32 = cache.cpu().float() if codes == "int8" else \
            cache.view(torch.uint8).cpu().contiguous().view(torch.float8_e4m3fn).float()
        values = (codes32 * scales[..., which].cpu().transpose(1, 2)[..., None]).to(dtype)
        want = torch.full((T, hkv, d), 3.0, dtype=dtype)
        for t in range(cu[0], cu[-1]):
            want[t] = 0 if where[t] is None else values[where[t]]
        assert torch.equal(out.cpu(), want)


def test_read_without_start_and_into_strides():
    g = gen_of(5)
    kc, vc, scales, kv, vv = filled(g, "e4m3", 4, 16, 2, 64)
    rows = torch.zeros(40, 6, 64, dtype=HF, device="cuda")
    k, v = rnn.kv_read_q8(kc, vc, scales, ints([[3, 1, 0]]), ints([0, 40]), 40, HF,
                          k_out=rows[:, 1:3], v_out=rows[:, 4:])
    a = rnn.kv_read_q8(kc, vc, scales, ints([[3, 1, 0]]), ints([0, 40]), 40, HF)
    assert torch.equal(k, a[0]) and torch.equal(v, a[1])
    assert (rows[:, 0] == 0).all() and (rows[:, 3] == 0).all()
    want = np.concatenate([kv[3], kv[1], kv[0]])[:40]
    assert np.all(np.abs(f64(k) - want) <= 2.0 ** -11 * np.abs(want) + 2.0 ** -25)


# ------------------------------------------------------------------ decode
def run_decode(codes, dtype, lens, hq, hkv, d, size, layout="plain", seed=0, std=1.0, spread=0.5,
               scale=None, change=None, q_strided=False):
    g = gen_of(seed)
    table, pages = deal(g, lens, size)
    kc, vc, scales, kv, vv = filled(g, codes, pages, size, hkv, d, layout, spread)
    if change:
        change(table, kc, vc, scales, kv, vv)
    B = len(lens)
    q = normal(g, (B, hq + 3, d + 8), dtype, std)[:, 2:2 + hq, 8:] if q_strided else \
        normal(g, (B, hq, d), dtype, std)
    out, lse = rnn.attn_decode_q8(q, kc, vc, scales, ints(table), ints(lens), scale=scale,
                                  with_lse=True)
    ref = oa.decode(f64(q), kv, vv, table, lens, 1 / math.sqrt(d) if scale is None else scale)
    check_attention_q8(out, lse, ref, dtype, d, np.abs(vv).max())
    return q, kc, vc, scales, table, out, lse


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d", [8, 24, 40, 64, 72, 96, 112, 128])
def test_decode_depths(codes, dtype, d):
    run_decode(codes, dtype, [70, 133, 1, 515], 4, 2, d, 16, seed=d)


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (8, 1), (9, 1), (16, 2), (17, 1), (40, 1), (6, 6), (32, 4)])
def test_decode_heads(codes, hq, hkv):
    run_decode(codes, BF, [45, 700], hq, hkv, 64, 16, seed=hq)
    run_decode(codes, HF, [45, 300], hq, hkv, 128, 24, seed=hq)


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
@pytest.mark.parametrize("size", [1, 3, 8, 16, 24, 48, 100, 128])
@pytest.mark.parametrize("layout", ["plain", "head", "wide"])
def test_decode_pages(codes, size, layout):
    run_decode(codes, HF, [0, 1, 15, 16, 17, 31, 33, 127, 128, 129, 400, 0], 4, 2, 64, size, layout,
               seed=size)
    run_decode(codes, BF, [0, 31, 32, 257], 4, 4, 72, size, layout, seed=size, q_strided=True)


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
def test_decode_many_sequences(codes):
    rng = np.random.default_rng(1)
    run_decode(codes, BF, rng.integers(0, 60, 500).tolist(), 2, 1, 32, 16)


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_long(codes, d):
    run_decode(codes, HF, [40000, 9], 2, 1, d, 64, seed=d)


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
def test_decode_pages_that_do_not_exist(codes):
    def change(table, kc, vc, scales, kv, vv):
        table[0, 1], table[0, 3], table[1, :] = -1, 99999, -5

    run_decode(codes, BF, [300, 100, 64], 4, 2, 128, 16, change=change)
    run_decode(codes, HF, [300, 100, 64], 4, 2, 64, 20, change=change)


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("spread", [3.0, 12.0])
def test_decode_values_of_very_different_size(codes, d, spread):
    """Scales over many powers of two, in keys and in values, in any order of the keys."""
    def change(table, kc, vc, scales, kv, vv):
        # keys as they would be without the spread: only the values' sizes differ
        k = scales[..., 0].clone()
        scales[..., 0] = k / k * 0.01
        kv /= k.double().cpu().numpy().transpose(0, 2, 1)[..., None]
        kv *= float(torch.tensor(0.01))

    run_decode(codes, BF, [800, 300], 4, 2, d, 16, seed=3, spread=spread, change=change)


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
@pytest.mark.parametrize("up", [True, False])
def test_decode_a_heavy_key_of_small_value(codes, up):
    """The weight of a value and the probability of its key at opposite ends."""
    d, n = 64, 600

    def change(table, kc, vc, scales, kv, vv):
        for b in range(1):
            for t in range(n):
                pg, row = table[b, t // 16], t % 16
                at = t / n if up else 1 - t / n
                f = np.float32(2.0 ** (40 * at - 30))
                g = np.float32(2.0 ** (-6 * at))
                for which, x, y in ((1, vv, f), (0, kv, g)):
                    scales[pg, :, row, which] *= float(y)
                    x[pg, row] *= float(y)

    run_decode(codes, BF, [n], 3, 1, d, 16, std=2.0, change=change)


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_growing_scores(codes, d):
    def change(table, kc, vc, scales, kv, vv):
        n = 900
        for t in range(n):
            pg, row = table[0, t // 16], t % 16
            f = np.float32(0.02 + 3 * t / n)
            scales[pg, :, row, 0] *= float(f)
            kv[pg, row] *= float(f)

    run_decode(codes, HF, [900], 2, 2, d, 16, change=change)


@pytest.mark.parametrize("std,scale", [(1e-6, None), (1e30, 1e-30), (3e-30, 1e30), (1.0, 40.0), (0.0, 1.0)])
def test_decode_queries_of_any_size(std, scale):
    run_decode("int8", BF, [50, 333], 4, 2, 64, 16, std=std, scale=scale)
    run_decode("e4m3", BF, [50, 333], 4, 1, 128, 16, std=std, scale=scale)


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_what_is_not_finite_shows(codes, d):
    g = gen_of(12)
    table, pages = deal(g, [300, 40], 16)
    kc, vc, scales, _, _ = filled(g, codes, pages, 16, 2, d)
    q = normal(g, (2, 4, d), BF)
    args = (kc, vc, scales, ints(table), ints([300, 40]))
    good, good_lse = rnn.attn_decode_q8(q, *args, with_lse=True)
    assert good.isfinite().all() and good_lse.isfinite().all()
    scales[table[0, 3], 1, 2, 0] = float("nan")            # one key of the second head
    out, lse = rnn.attn_decode_q8(q, *args, with_lse=True)
    assert torch.equal(out[1], good[1]) and torch.equal(out[0, :2], good[0, :2])
    assert out[0, 2:].isnan().all() and lse[0, 2:].isnan().all()
    scales[table[0, 3], 1, 2, 0] = 1.0
    scales[table[1, 0], 0, 2, 1] = float("nan")            # one value of the first head
    out = rnn.attn_decode_q8(q, *args)
    assert out[1, :2].isnan().all() and out[1, 2:].isfinite().all() and out[0].isfinite().all()
    scales[table[1, 0], 0, 2, 1] = 1.0
    q[0, 1, 5], q[1, 3, 7] = float("nan"), float("inf")
    out = rnn.attn_decode_q8(q, *args)
    assert out[0, 1].isnan().all() and out[1, 3].isnan().all()
    assert out[0, 0].isfinite().all() and out[0, 2:].isfinite().all() and out[1, :3].isfinite().all()


def test_decode_rows_behind_the_last_key_may_hold_anything():
    g = gen_of(2)
    lens = [37, 100]
    table, pages = deal(g, lens, 32)
    kc, vc, scales, _, _ = filled(g, "e4m3", pages, 32, 2, 64)
    q = normal(g, (2, 4, 64), HF)
    want = rnn.attn_decode_q8(q, kc, vc, scales, ints(table), ints(lens))
    for b, n in enumerate(lens):
        kc.view(torch.uint8)[table[b, n // 32], n % 32:] = 0x7F
        vc.view(torch.uint8)[table[b, n // 32], n % 32:] = 0x7F
        scales[table[b, n // 32], :, n % 32:] = float("inf")
    assert torch.equal(rnn.attn_decode_q8(q, kc, vc, scales, ints(table), ints(lens)), want)


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
def test_decode_long_tables(codes):
    """The form for tables with room for many keys, over more keys than one accumulator takes."""
    g = gen_of(9)
    n, size, d = 300000, 256, 64
    table, pages = deal(g, [n], size)
    kc = torch.randint(-100, 101, (pages, size, 1, d), device="cuda", dtype=torch.int32)
    vc = torch.randint(20, 101, (pages, size, 1, d), device="cuda", dtype=torch.int32)
    kc, vc = (x.to(torch.int8) if codes == "int8" else x.float().to(CODES[codes]) for x in (kc, vc))
    scales = torch.rand(pages, 1, size, 2, device="cuda") * 0.01 + 0.001
    q = normal(g, (1, 2, d), HF)
    out, lse = rnn.attn_decode_q8(q, kc, vc, scales, ints(table), ints([n]), with_lse=True)
    dec = [(x.float() if codes == "int8" else x.view(torch.uint8).view(CODES[codes]).float()).double()
           * scales[..., w].transpose(1, 2)[..., None].double() for w, x in enumerate((kc, vc))]
    ref = oa.decode(f64(q), f64(dec[0]), f64(dec[1]), table, [n], 1 / 8)
    # each sum leaves its accumulator every 65536 keys: 2^-11 of it may be cut off
    ref.spread *= 1 + 2.0 ** -11 / 2.0 ** -12
    check_attention_q8(out, lse, ref, HF, d, float(dec[1].max()))


# --------------------------------------------------------------- as it is used
@pytest.mark.parametrize("codes", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_append_decode_and_read_back_together(codes, dtype):
    """A prompt goes in, is continued token by token, and is read back for the next prompt."""
    g = gen_of(11)
    B, hq, hkv, d, size = 3, 4, 2, 64, 16
    new = [40, 7, 100]
    steps = 3
    table, pages = deal(g, [n + steps for n in new], size)
    table_t = ints(table)
    kc, vc, scales = new_cache(codes, pages, size, hkv, d)
    inv = (10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)).cuda()
    lens = list(new)
    q, k, v = (normal(g, (sum(new), h, d), dtype) for h in (hq, hkv, hkv))
    rnn.kv_append_q8(k, v, kc, vc, scales, table_t, ints([0] * B), ints(cum(new)), q=q, inv_freq=inv)
    for _ in range(steps):
        q, k, v = (normal(g, (B, h, d), dtype) for h in (hq, hkv, hkv))
        qr, _ = rnn.kv_append_q8(k, v, kc, vc, scales, table_t, ints(lens), ints(range(B + 1)), q=q,
                                 inv_freq=inv)
        lens = [n + 1 for n in lens]
        out, lse = rnn.attn_decode_q8(qr, kc, vc, scales, table_t, ints(lens), with_lse=True)
        values = [oq.value(raw(c), codes) * f64(scales)[..., w].transpose(0, 2, 1)[..., None]
                  for w, c in enumerate((kc, vc))]
        ref = oa.decode(f64(qr), *values, table, lens, d ** -0.5)
        vmax = max(np.abs(values[1][table[b, :-(-n // size)]]).max() for b, n in enumerate(lens))
        check_attention_q8(out, lse, ref, dtype, d, vmax)
    # the last tokens' rows through attn_prompt over what is read back
    ka, va = rnn.kv_read_q8(kc, vc, scales, table_t, ints(cum(lens)), sum(lens), dtype)
    again = rnn.attn_prompt(qr, ka, va, ints(range(B + 1)), ints(cum(lens)))
    # keys, values (1.5 steps with the weights) and outputs rounded to 16 bits: a score moves by
    # u reach, the output by 2 u reach and 4 u of the weighted |values|
    u = torch.finfo(dtype).eps / 2
    tol = (2 * u * ref.reach[..., None] * 1.1 + 4 * u) * ref.spread + u * np.abs(ref.out) + 1e-5
    assert np.all(np.abs(f64(again) - ref.out) <= tol)


def test_graph_streams_and_a_given_workspace():
    """Captured and replayed with new inputs, on another stream than the tensors' own."""
    g = gen_of(4)
    B, hq, hkv, d, size = 5, 4, 2, 128, 16
    lens = [100, 3, 250, 0, 64]
    table, pages = deal(g, [n + 1 for n in lens], size)
    kc, vc, scales, _, _ = filled(g, "e4m3", pages, size, hkv, d)
    keep = [x.clone() for x in (kc.view(torch.uint8), vc.view(torch.uint8), scales)]
    inv = torch.ones(64, dtype=torch.float64, device="cuda")
    q, k, v = (normal(g, (B, h, d), BF) for h in (hq, hkv, hkv))
    tab, start, now, cu = ints(table), ints(lens), ints([n + 1 for n in lens]), ints(range(B + 1))
    ws = torch.empty(rnn.cache_q8._decode_need(B, hq, hkv, d), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)

    def step():
        qr, _ = rnn.kv_append_q8(k, v, kc, vc, scales, tab, start, cu, q=q, inv_freq=inv)
        rnn.attn_decode_q8(qr, kc, vc, scales, tab, now, out=out, workspace=ws)
        return rnn.kv_read_q8(kc, vc, scales, tab, cu, B, BF, start=start)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        read = step()
    for seed in (1, 2):
        gg = gen_of(seed)
        for t in (q, k, v):
            t.copy_(normal(gg, tuple(t.shape), BF))
        for t, old in zip((kc.view(torch.uint8), vc.view(torch.uint8), scales), keep):
            t.copy_(old)
        graph.replay()
        torch.cuda.synchronize()
        rnn.workspace_status(ws)
        got = [out.clone(), *(x.clone() for x in read), kc.view(torch.uint8).clone(), scales.clone()]
        for t, old in zip((kc.view(torch.uint8), vc.view(torch.uint8), scales), keep):
            t.copy_(old)
        out.zero_()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            again = step()
        side.synchronize()
        for a, b in zip(got, [out, *again, kc.view(torch.uint8), scales]):
            assert torch.equal(a, b)


def test_nothing_to_do():
    kc, vc, scales = new_cache("int8", 2, 4, 2, 64)
    z = torch.zeros(0, 2, 64, dtype=BF, device="cuda")
    assert rnn.kv_append_q8(z, z, kc, vc, scales, ints([[0]]), ints([0]), ints([0, 0])) == (None, None)
    k, v = rnn.kv_read_q8(kc, vc, scales, ints([[0]]), ints([0, 0]), 0, BF)
    assert k.shape == v.shape == (0, 2, 64)
    none = torch.zeros(0, 1, dtype=torch.int32, device="cuda")
    assert rnn.attn_decode_q8(z, kc, vc, scales, none, ints([])).shape == (0, 2, 64)
    x = torch.ones(3, 2, 64, dtype=BF, device="cuda")
    out = rnn.kv_read_q8(kc, vc, scales, none, ints([0]), 3, BF, k_out=x)[0]
    assert (out == 1).all()
    assert (raw(kc) == 0x5A).all() and (scales == 7).all()


def test_python_forms_give_the_same(monkeypatch):
    """The calls' way through the extension module and the one through Python."""
    g = gen_of(6)
    lens, size, d = [37, 100], 16, 64
    table, pages = deal(g, [n + 1 for n in lens], size)
    kc, vc, scales, _, _ = filled(g, "e4m3", pages, size, 2, d)
    q, k, v = (normal(g, (2, h, d), HF) for h in (4, 2, 2))
    inv = torch.ones(32, dtype=torch.float64, device="cuda")
    tab, now, cu = ints(table), ints(lens), ints([0, 1, 2])

    def everything():
        a = rnn.kv_append_q8(k, v, kc, vc, scales, tab, now, cu, q=q, inv_freq=inv, with_k=True)
        b = rnn.kv_read_q8(kc, vc, scales, tab, ints(cum(lens)), sum(lens), HF)
        c = rnn.attn_decode_q8(a[0], kc, vc, scales, tab, now, with_lse=True, scale=0.25)
        return *a, *b, *c, kc.view(torch.uint8).clone(), scales.clone()

    assert rnn._lib.load_fast().__name__.endswith("_fast")
    mine = everything()
    monkeypatch.setattr(rnn._lib, "fast", rnn._lib._Python)
    for x, y in zip(mine, everything()):
        assert torch.equal(x, y) and x.dtype == y.dtype and x.stride() == y.stride()


def test_a_size_of_one_may_have_any_stride():
    g = gen_of(6)
    kc, vc, scales, kv, vv = filled(g, "int8", 3, 16, 1, 64)
    kc, vc = (x.as_strided((3, 16, 1, 64), (1024, 64, 3, 1)) for x in (kc, vc))
    q = normal(g, (1, 2, 64), HF).as_strided((1, 2, 64), (5, 64, 1))
    out, lse = rnn.attn_decode_q8(q, kc, vc, scales, ints([[2, 0]]), ints([20]), with_lse=True)
    ref = oa.decode(f64(q), kv, vv, np.array([[2, 0]]), [20], 1 / 8)
    check_attention_q8(out, lse, ref, HF, 64, np.abs(vv).max())


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
def test_offsets_beyond_32_bits(codes):
    """Pages 1.5 10^9 codes apart, and scales 6 10^8 floats."""
    g = gen_of(1)
    d, size, hkv, gap = 64, 16, 2, 1500000000 // 16 * 16
    store = torch.zeros(4 * gap, dtype=torch.uint8, device="cuda")
    shape, strides = (4, size, hkv, d), (gap, hkv * d, d, 1)
    kc, vc = (store[o:].as_strided(shape, strides).view(CODES[codes]) for o in (0, gap // 2 // 16 * 16))
    scale_gap = 600000000
    scales = torch.zeros(4 * scale_gap, device="cuda").as_strided((4, hkv, size, 2), (scale_gap, 2 * size, 2, 1))
    lens = [40, 16]
    table = np.array([[3, 0, 2], [1, -1, -1]])
    k, v = (normal(g, (56, hkv, d), HF) for _ in range(2))
    args = (kc, vc, scales, ints(table))
    rnn.kv_append_q8(k, v, *args, ints([0, 0]), ints([0, 40, 56]))
    values = []
    for x in (k, v):
        c, s = oq.quantise32(x.float().cpu().numpy(), codes)
        values.append(c * s[..., None].astype(np.float64))
    got = rnn.kv_read_q8(*args, ints([0, 40, 56]), 56, HF)
    for x, y in zip(got, values):
        assert np.all(np.abs(f64(x) - y) <= 2.0 ** -11 * np.abs(y) + 2.0 ** -25)
    q = normal(g, (2, 4, d), HF)
    out, lse = rnn.attn_decode_q8(q, *args, ints(lens), with_lse=True)
    packed = [np.zeros((4, size, hkv, d)) for _ in range(2)]
    for b, n in enumerate(lens):
        for t in range(n):
            for to, x in zip(packed, values):
                to[table[b, t // size], t % size] = x[(0, 40)[b] + t]
    ref = oa.decode(f64(q), *packed, table, lens, 1 / 8)
    check_attention_q8(out, lse, ref, HF, d, np.abs(packed[1]).max())


def test_many_empty_sequences_and_the_same_page_twice():
    g = gen_of(7)
    lens = [0] * 300 + [5] + [0] * 400 + [33, 0, 1]
    table, pages = deal(g, lens, 16)
    table[-1, 0] = table[300, 0]                  # two sequences on one page
    kc, vc, scales, kv, vv = filled(g, "int8", pages, 16, 2, 64)
    cu = cum(lens)
    got = rnn.kv_read_q8(kc, vc, scales, ints(table), ints(cu), cu[-1], HF)
    where, _ = oa.slots(cu, [0] * len(lens), table, 16, pages, cu[-1])
    for x, y in zip(got, (kv, vv)):
        want = np.stack([y[w] for w in where])
        assert np.all(np.abs(f64(x) - want) <= 2.0 ** -11 * np.abs(want) + 2.0 ** -25)
    q = normal(g, (len(lens), 4, 64), HF)
    out, lse = rnn.attn_decode_q8(q, kc, vc, scales, ints(table), ints(lens), with_lse=True)
    ref = oa.decode(f64(q), kv, vv, table, lens, 1 / 8)
    check_attention_q8(out, lse, ref, HF, 64, np.abs(vv).max())


def test_many_tokens_read():
    """Enough of them that a warp takes several."""
    g = gen_of(8)
    lens = [25000, 1, 0, 14000, 3]
    table, pages = deal(g, lens, 64)
    kc, vc, scales, _, _ = filled(g, "e4m3", pages, 64, 1, 16)
    cu = cum(lens)
    k, v = rnn.kv_read_q8(kc, vc, scales, ints(table), ints(cu), cu[-1] + 5, BF,
                          k_out=torch.full((cu[-1] + 5, 1, 16), 3.0, dtype=BF, device="cuda"))
    assert (k[cu[-1]:] == 3).all()
    number = np.concatenate([np.arange(n) for n in lens])
    seq = np.repeat(np.arange(len(lens)), lens)
    page, row = torch.from_numpy(table[seq, number // 64]).cuda(), torch.from_numpy(number % 64).cuda()
    for which, (out, cache) in enumerate(((k, kc), (v, vc))):
        want = cache.view(torch.uint8)[page, row].view(CODES["e4m3"]).float() * \
            scales[..., which].transpose(1, 2)[page, row][..., None]
        assert torch.equal(out[:cu[-1]], want.to(BF))


def test_two_calls_at_once():
    g = gen_of(4)
    lens = [700, 3, 90, 2000]
    table, pages = deal(g, lens, 16)
    sets = []
    for s in (1, 2):
        kc, vc, scales, _, _ = filled(gen_of(s), "e4m3", pages, 16, 2, 128)
        sets.append((normal(g, (4, 8, 128), BF), kc, vc, scales, ints(table), ints(lens)))
    want = [rnn.attn_decode_q8(*a) for a in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(rnn.attn_decode_q8(*sets[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])


def test_refusals_reach_the_caller():
    """Through the extension module as through Python."""
    g = gen_of(3)
    kc, vc, scales, _, _ = filled(g, "int8", 3, 16, 2, 64)
    q = normal(g, (1, 4, 64), HF)
    tab, lens = ints([[0, 1]]), ints([20])
    with pytest.raises(TypeError):
        rnn.attn_decode_q8(q, kc.view(CODES["e4m3"]), vc, scales, tab, lens)
    with pytest.raises(ValueError):
        rnn.attn_decode_q8(q, kc, vc, scales[:2], tab, lens)
    with pytest.raises(ValueError):
        rnn.attn_decode_q8(q, kc, vc, scales, tab, lens, scale=-1.0)
    with pytest.raises(rnn.RNNError) as e:
        rnn.attn_decode_q8(q, kc, vc, scales, tab, lens, workspace=torch.empty(
            256, dtype=torch.uint8, device="cuda"))
    assert e.value.name == "RNN_EWORKSPACE"
    two = torch.zeros(2, 4, 64, dtype=HF, device="cuda")
    with pytest.raises(rnn.RNNError) as e:          # rows of the output that overlap
        rnn.attn_decode_q8(two, kc, vc, scales, ints([[0, 1]] * 2), ints([20, 3]),
                           out=two.new_zeros(1024).as_strided((2, 4, 64), (64, 64, 1)))
    assert e.value.name == "RNN_EINVAL"
    k = normal(g, (5, 2, 64), HF)
    with pytest.raises(rnn.RNNError):               # the same output twice
        rnn.kv_read_q8(kc, vc, scales, tab, ints([0, 5]), 5, HF, k_out=k, v_out=k)
    with pytest.raises(ValueError):
        rnn.kv_append_q8(k, k, kc, vc, scales, tab, ints([0]), ints([0, 5]), q=k)
