"""Attention operators against the double-precision oracle (needs a B200)."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import reciprocal_nearest_neighbour_b200 as rnn
from attn_bounds import check_attention
from oracle import attention as oa

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def f64(t):
    return t.double().cpu().numpy()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cum(lens):
    return [0] + np.cumsum(lens).tolist()


def normal(gen, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=gen, dtype=torch.float32) * std).to(dtype).cuda()


def gen_of(seed):
    return torch.Generator().manual_seed(seed)


# ------------------------------------------------------------------ prompts
def run_prompt(dtype, nq, nk, hq, hkv, d, causal, seed, std=1.0, front=0, behind=0, layout="thd"):
    """Packed sequences with `front` and `behind` rows outside them that hold NaN."""
    g = gen_of(seed)
    tq, tk = sum(nq) + front + behind, sum(nk) + front + behind

    def rows(t, h):
        if layout == "htd":     # heads outermost
            return normal(g, (h, t, d), dtype, std).transpose(0, 1)
        if layout == "fused":   # a slice of a wider row
            return normal(g, (t, h + 2, d + 8), dtype, std)[:, 1:1 + h, 8:]
        return normal(g, (t, h, d), dtype, std)

    q, k, v = rows(tq, hq), rows(tk, hkv), rows(tk, hkv)
    cu_q = [front + x for x in cum(nq)]
    cu_k = [front + x for x in cum(nk)]
    for t, cu in ((q, cu_q), (k, cu_k), (v, cu_k)):
        t[:cu[0]] = float("nan")
        t[cu[-1]:] = float("nan")
    out = torch.full((tq, hq, d), 7.0, dtype=dtype, device="cuda")
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    got, lse = rnn.attn_prompt(q, k, v, ints(cu_q), ints(cu_k), causal=causal, with_lse=True,
                               out=out, workspace=ws)
    rnn.workspace_status(ws)
    assert got is out
    assert (out[:cu_q[0]] == 7).all() and (out[cu_q[-1]:] == 7).all()
    ref = oa.prompt(f64(q), f64(k), f64(v), cu_q, cu_k, causal, 1 / math.sqrt(d))
    live = slice(cu_q[0], cu_q[-1])
    for f in ("out", "lse", "spread", "reach", "keys"):
        setattr(ref, f, getattr(ref, f)[live])
    vmax = float(v[cu_k[0]:cu_k[-1]].float().abs().max()) if sum(nk) else 0.0
    check_attention(out[live], lse[live], ref, dtype, d, vmax)
    return q, k, v, cu_q, cu_k, out, lse


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d", [8, 24, 40, 64, 72, 96, 112, 128])
def test_prompt_depths(dtype, d):
    run_prompt(dtype, [70, 133], [70, 133], 2, 1, d, True, d)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (3, 3), (4, 2), (6, 2), (5, 1), (8, 1)])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_heads(hq, hkv, causal):
    run_prompt(BF, [200, 40], [200, 40], hq, hkv, 64, causal, 10 * hq + hkv)


@pytest.mark.parametrize("n", [1, 2, 127, 128, 129, 255, 256, 257, 500])
@pytest.mark.parametrize("hq", [1, 2])
def test_prompt_lengths(n, hq):
    run_prompt(HF, [n], [n], hq, 1, 64, True, n)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hkv", [1, 2])
def test_prompt_ragged(causal, d, hkv):
    """Empty sequences, sequences without keys, more and fewer keys than queries."""
    nq = [0, 5, 1, 0, 130, 300, 17, 64, 0]
    nk = [3, 5, 0, 0, 700, 41, 18, 640, 9]
    run_prompt(BF, nq, nk, 2, hkv, d, causal, 5, front=3, behind=150)


@pytest.mark.parametrize("layout", ["htd", "fused"])
@pytest.mark.parametrize("d", [64, 96])
def test_prompt_strides(layout, d):
    run_prompt(HF, [150, 31], [150, 31], 4, 2, d, True, 8, layout=layout)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_prompt_many_sequences(dtype):
    rng = np.random.default_rng(4)
    nq = rng.integers(0, 6, 700).tolist()
    run_prompt(dtype, nq, [n + 1 for n in nq], 2, 1, 32, True, 9)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_growing_scores(dtype, d):
    """Every key tile's scores exceed the last one's, so every tile rescales."""
    g = gen_of(3)
    n = 640
    q = normal(g, (n, 2, d), dtype, 0.5) + 1.0
    ramp = torch.linspace(-8, 8, n)[:, None, None].cuda()
    k = (normal(g, (n, 1, d), dtype, 0.1).float() + ramp).to(dtype)
    v = normal(g, (n, 1, d), dtype)
    for causal in (True, False):
        out, lse = rnn.attn_prompt(q, k, v, ints([0, n]), causal=causal, with_lse=True)
        ref = oa.prompt(f64(q), f64(k), f64(v), [0, n], [0, n], causal, 1 / math.sqrt(d))
        check_attention(out, lse, ref, dtype, d, float(v.abs().max()))


@pytest.mark.parametrize("dtype", [BF, HF])
def test_prompt_one_key_takes_all(dtype):
    """Weights from 1 down to far below the 16-bit types' range, values of one sign."""
    g = gen_of(6)
    n, d = 400, 64
    q = normal(g, (n, 2, d), dtype) * 0.1 + 1.0
    k = normal(g, (n, 2, d), dtype) * 0.1
    k[n // 2] += 2.0
    v = normal(g, (n, 2, d), dtype).abs() + 0.5
    out, lse = rnn.attn_prompt(q, k, v, ints([0, n]), causal=False, scale=1.0, with_lse=True)
    ref = oa.prompt(f64(q), f64(k), f64(v), [0, n], [0, n], False, 1.0)
    check_attention(out, lse, ref, dtype, d, float(v.abs().max()))


def test_prompt_neighbours_do_not_leak():
    """A sequence's rows do not depend on what the next sequence holds."""
    g = gen_of(7)
    n, d = 77, 128
    q, k, v = (normal(g, (2 * n, 2, d), BF) for _ in range(3))
    for causal in (True, False):
        a = rnn.attn_prompt(q, k, v, ints([0, n, 2 * n]), causal=causal)[:n].clone()
        for t in (q, k, v):
            t[n:] = float("inf")
        b = rnn.attn_prompt(q, k, v, ints([0, n, 2 * n]), causal=causal)[:n]
        assert torch.equal(a, b)
        for t in (q, k, v):
            t[n:] = 0


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_prompt_bad_scores_show(dtype, d, bad):
    """A score that is not a number makes the rows that see it NaN, and no others."""
    g = gen_of(12)
    n, at = 300, 140
    q = normal(g, (n, 4, d), dtype)
    q[:, :, 0] = 1.0                  # so that the score of an infinite key is infinite
    k, v = (normal(g, (n, 2, d), dtype) for _ in range(2))
    good, good_lse = rnn.attn_prompt(q, k, v, ints([0, n]), with_lse=True)
    k[at, 1, 0] = bad
    out, lse = rnn.attn_prompt(q, k, v, ints([0, n]), with_lse=True)
    assert torch.equal(out[:, :2], good[:, :2]) and torch.equal(lse[:, :2], good_lse[:, :2])
    assert torch.equal(out[:at], good[:at]) and torch.equal(lse[:at], good_lse[:at])
    assert out[at:, 2:].isnan().all() and lse[at:, 2:].isnan().all()
    k[:, 1, 0] = float("nan")         # rows without a single number
    out, lse = rnn.attn_prompt(q, k, v, ints([0, n]), causal=False, with_lse=True)
    assert out[:, 2:].isnan().all() and lse[:, 2:].isnan().all()
    assert out[:, :2].isfinite().all() and lse[:, :2].isfinite().all()


def test_prompt_nothing_to_do():
    z = torch.zeros((0, 2, 64), dtype=BF, device="cuda")
    kv = torch.zeros((5, 2, 64), dtype=BF, device="cuda")
    assert rnn.attn_prompt(z, kv, kv, ints([0, 0]), ints([0, 5])).shape == (0, 2, 64)
    q = torch.ones((4, 2, 64), dtype=BF, device="cuda")
    out, lse = rnn.attn_prompt(q, z, z, ints([0, 4]), ints([0, 0]), with_lse=True)
    assert (out == 0).all() and torch.isneginf(lse).all()
    out = rnn.attn_prompt(q, kv, kv, ints([0]), ints([0]), out=q.clone())
    assert (out == 1).all()


def test_prompt_bad_offsets_stay_in_bounds():
    """Offsets that fall or leave the tensors give some rows, and no access outside."""
    q = normal(gen_of(1), (50, 2, 64), BF)
    for cu in ([0, 400], [-7, 50], [40, 10, 50], [60, 90]):
        out = torch.zeros_like(q)
        rnn.attn_prompt(q, q, q, ints(cu), out=out)
        torch.cuda.synchronize()
        assert torch.isfinite(out.float()).all()


def test_prompt_wait_runs_out_and_is_reported():
    q = normal(gen_of(2), (100, 2, 64), BF)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    lib = rnn._lib.load()
    lib.rnn_test_stall_loads(1, 50_000_000)
    try:
        rnn.attn_prompt(q, q, q, ints([0, 100]), workspace=ws)
        torch.cuda.synchronize()
    finally:
        lib.rnn_test_stall_loads(0, 0)
    with pytest.raises(rnn.RNNError) as e:
        rnn.workspace_status(ws)
    assert e.value.name == "RNN_ETIMEOUT"
    out, lse = rnn.attn_prompt(q, q, q, ints([0, 100]), with_lse=True, workspace=ws)
    rnn.workspace_status(ws)
    ref = oa.prompt(f64(q), f64(q), f64(q), [0, 100], [0, 100], True, 1 / 8)
    check_attention(out, lse, ref, BF, 64, float(q.abs().max()))


# ------------------------------------------------------------------- decode
def paged(gen, lens, size, hkv, d, dtype, order="phsd"):
    """Caches full of NaN but for the sequences' rows, and the page table."""
    need = [-(-max(n, 0) // size) for n in lens]
    count = sum(need) + 2
    deal = torch.randperm(count, generator=gen).tolist()
    table = np.full((len(lens), max(need + [1]) + 1), -9, dtype=np.int32)
    shape = {"phsd": (count, size, hkv, d), "pshd": (count, hkv, size, d)}[order]
    caches = []
    for _ in range(2):
        c = torch.full(shape, float("nan"), dtype=dtype, device="cuda")
        caches.append(c if order == "phsd" else c.transpose(1, 2))
    at = 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = deal[at:at + need[b]]
        at += need[b]
        for i in range(need[b]):
            rows = min(size, n - i * size)
            for c in caches:
                c[int(table[b, i]), :rows] = normal(gen, (rows, hkv, d), dtype)
    return caches[0], caches[1], table


def run_decode(dtype, lens, size, hq, hkv, d, seed, order="phsd"):
    g = gen_of(seed)
    kc, vc, table = paged(g, lens, size, hkv, d, dtype, order)
    q = normal(g, (len(lens), hq, d), dtype)
    out, lse = rnn.attn_decode(q, kc, vc, torch.from_numpy(table).cuda(), ints(lens),
                               with_lse=True)
    ref = oa.decode(f64(q), f64(kc), f64(vc), table, lens, 1 / math.sqrt(d))
    check_attention(out, lse, ref, dtype, d, 6.0)
    return q, kc, vc, table, out, lse


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d", [8, 24, 40, 64, 72, 96, 112, 128])
def test_decode_depths(dtype, d):
    run_decode(dtype, [1, 100, 37], 16, 4, 2, d, d)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 3), (8, 1), (12, 2), (16, 1), (17, 1), (40, 2),
                                    (64, 1)])
def test_decode_heads(hq, hkv):
    run_decode(BF, [130, 5], 16, hq, hkv, 64, hq)


@pytest.mark.parametrize("size", [1, 7, 16, 48, 64, 100, 256])
def test_decode_pages(size):
    run_decode(HF, [0, 1, 15, 16, 17, 63, 64, 65, 301], size, 4, 2, 64, size)


@pytest.mark.parametrize("order", ["phsd", "pshd"])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_long(order, d):
    """Few sequences, so each is split over many blocks and joined."""
    run_decode(BF, [5000], 64, 2, 1, d, 3, order)
    run_decode(BF, [2777, 0, 901], 16, 8, 1, d, 4, order)


def test_decode_many_sequences():
    rng = np.random.default_rng(5)
    lens = rng.integers(-2, 40, 900).tolist()
    run_decode(BF, lens, 8, 2, 1, 32, 6)


def test_decode_lengths_beyond_the_table():
    g = gen_of(8)
    kc, vc, table = paged(g, [32, 20], 16, 1, 64, BF)
    q = normal(g, (2, 2, 64), BF)
    table = np.ascontiguousarray(table[:, :2])
    out = rnn.attn_decode(q, kc, vc, torch.from_numpy(table).cuda(), ints([2000000000, 20]))
    ref = oa.decode(f64(q), f64(kc), f64(vc), table, [32, 20], 1 / 8)
    check_attention(out, None, ref, BF, 64, 6.0)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("lens", [[70, 33], [4000, 90]])   # pairs in one share, and joined
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_decode_bad_scores_show(dtype, lens, bad):
    g = gen_of(13)
    kc, vc, table = paged(g, lens, 16, 2, 64, dtype)
    q = normal(g, (2, 4, 64), dtype)
    q[:, :, 0] = 1.0
    t = torch.from_numpy(table).cuda()
    good, good_lse = rnn.attn_decode(q, kc, vc, t, ints(lens), with_lse=True)
    kc[int(table[0, 3]), 5, 1, 0] = bad           # token 53 of the first sequence
    out, lse = rnn.attn_decode(q, kc, vc, t, ints(lens), with_lse=True)
    for b, h in ((0, 0), (0, 1), (1, 0), (1, 1), (1, 2), (1, 3)):
        assert torch.equal(out[b, h], good[b, h]) and torch.equal(lse[b, h], good_lse[b, h])
    assert out[0, 2:].isnan().all() and lse[0, 2:].isnan().all()
    kc[:, :, 1, 0] = float("nan")
    out, lse = rnn.attn_decode(q, kc, vc, t, ints(lens), with_lse=True)
    assert out[:, 2:].isnan().all() and lse[:, 2:].isnan().all()
    assert torch.equal(out[:, :2], good[:, :2]) and torch.equal(lse[:, :2], good_lse[:, :2])


def test_decode_missing_pages():
    g = gen_of(9)
    kc, vc, table = paged(g, [200, 48, 16], 16, 2, 64, HF)
    table[0, 3] = -1
    table[0, 7] = kc.shape[0]
    table[0, 8] = 2000000000
    table[1, :3] = -5            # a sequence without a single page
    q = normal(g, (3, 4, 64), HF)
    out, lse = rnn.attn_decode(q, kc, vc, torch.from_numpy(table).cuda(), ints([200, 48, 16]),
                               with_lse=True)
    ref = oa.decode(f64(q), f64(kc), f64(vc), table, [200, 48, 16], 1 / 8)
    assert ref.keys[0, 0] == 152 and ref.keys[1, 0] == 0
    check_attention(out, lse, ref, HF, 64, 6.0)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_decode_many_small_weights(dtype):
    """One key far above thousands of others whose values have one sign."""
    g = gen_of(10)
    n, d = 6000, 64
    kc, vc, table = paged(g, [n], 64, 1, d, dtype)
    q = normal(g, (1, 2, d), dtype) * 0.05 + 1.0
    kc.mul_(0.02)
    vc.abs_().add_(0.5)
    kc[int(table[0, 3]), 7] += 14.0 / d
    out, lse = rnn.attn_decode(q, kc, vc, torch.from_numpy(table).cuda(), ints([n]), scale=1.0,
                               with_lse=True)
    ref = oa.decode(f64(q), f64(kc), f64(vc), table, [n], 1.0)
    check_attention(out, lse, ref, dtype, d, 6.5)


# ------------------------------------------------------------------- append
def run_append(dtype, lens, past, size, hq, hkv, d, pairs, axes, paired, seed, rotate=True,
               behind=0, layout="thd"):
    g = gen_of(seed)
    T = sum(lens) + behind
    totals = [a + b for a, b in zip(lens, past)]
    kc, vc, table = paged(g, totals, size, hkv, d, dtype)
    kc.copy_(normal(g, kc.shape, dtype))
    vc.copy_(normal(g, vc.shape, dtype))
    old_k, old_v = f64(kc), f64(vc)
    rows = normal(g, (T, hq + 2 * hkv, d), dtype)
    q, k, v = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]
    if layout == "htd":
        q, k, v = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v))
    cu = cum(lens)
    inv = 10000.0 ** (-np.arange(pairs) / max(pairs, 1))
    pos = None
    if axes == 2:
        pos = torch.randint(-3, 70000, (T, 2), generator=g, dtype=torch.int32).cuda()
    q_out = torch.full((T, hq, d), 7.0, dtype=dtype, device="cuda") if rotate and hq else None
    k_out = torch.full((T, hkv, d), 7.0, dtype=dtype, device="cuda")
    kw = dict(q=q, inv_freq=torch.from_numpy(inv).cuda(), positions=pos, paired=paired,
              q_out=q_out) if rotate else {}
    got_q, got_k = rnn.kv_append(k, v, kc, vc, torch.from_numpy(table).cuda(), ints(past),
                                 ints(cu), k_out=k_out, **kw)
    assert got_k is k_out and got_q is q_out
    where, number = oa.slots(cu, past, table, size, kc.shape[0], T)
    live = slice(0, cu[-1])
    place = f64(pos)[live] if pos is not None else np.array(number[live], float)[:, None]
    u = torch.finfo(dtype).eps / 2

    def check(got, x):
        # u |y| for the rounding; 2^-21 (|x1| + |x2|) for an angle good to 2^-23,
        # cos and sin to 2^-22 and fp32 products; |x1| + |x2| <= sqrt(2) |(x1, x2)|
        x = f64(x)[live]
        want = oa.rotate(x, place, inv, paired) if rotate else x
        size_ = np.abs(x).max(-1, keepdims=True) * 2 if rotate else 0
        tol = u * np.abs(want) * (1 if rotate else 0) + 2.0 ** -21 * size_ + \
            (2.0 ** -25 if rotate else 0)
        assert np.all(np.abs(got - want) <= tol), np.abs(got - want).max()
        rest = slice(2 * pairs * axes, None) if rotate else slice(0, None)
        assert np.array_equal(got[..., rest], x[..., rest])     # passed through

    if got_q is not None:
        check(f64(got_q)[live], q)
        assert (got_q[cu[-1]:] == 7).all()
    check(f64(got_k)[live], k)
    assert (k_out[cu[-1]:] == 7).all()
    new_k, new_v = f64(kc), f64(vc)
    packed_k, packed_v = f64(k_out), f64(v)
    for t, at in enumerate(where):
        if at is not None:
            assert np.array_equal(new_k[at], packed_k[t])       # the same bits as packed
            assert np.array_equal(new_v[at], packed_v[t])
            new_k[at], new_v[at] = old_k[at], old_v[at]
    assert np.array_equal(new_k, old_k) and np.array_equal(new_v, old_v)  # and nothing else


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("paired", [False, True])
@pytest.mark.parametrize("d,pairs,axes", [(64, 32, 1), (64, 16, 2), (128, 64, 1), (128, 32, 1),
                                          (40, 20, 1), (72, 18, 2), (24, 3, 2), (8, 4, 1),
                                          (96, 5, 1), (256, 128, 1)])
def test_append_rotations(dtype, paired, d, pairs, axes):
    run_append(dtype, [5, 0, 20], [3, 9, 0], 16, 4, 2, d, pairs, axes, paired, d + pairs)


@pytest.mark.parametrize("size", [1, 7, 16, 48, 256])
@pytest.mark.parametrize("layout", ["thd", "htd"])
def test_append_pages(size, layout):
    run_append(HF, [1, 40, 0, 17, 3], [0, 5, 100, 15, 16], size, 3, 1, 64, 32, 1, False, size,
               behind=9, layout=layout)


def test_append_without_rotation():
    run_append(BF, [3, 30], [2, 1], 16, 0, 2, 64, 0, 0, False, 2, rotate=False, behind=2)


def test_append_many_sequences():
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 4, 1500).tolist()
    past = rng.integers(0, 30, 1500).tolist()
    run_append(BF, lens, past, 8, 2, 1, 16, 8, 1, True, 5, behind=1)


def test_append_many_tokens():
    """Several tokens a block."""
    run_append(BF, [9000, 5800], [1, 70], 64, 1, 1, 16, 8, 1, False, 6, behind=3)


def test_append_far_positions():
    """Angles at positions where 32 bits would lose them."""
    d, pairs = 64, 32
    g = gen_of(4)
    k = normal(g, (3, 1, d), BF)
    pos = [2 ** 31 - 1, 1048577, -2 ** 31]
    kc = torch.zeros((1, 4, 1, d), dtype=BF, device="cuda")
    inv = 10000.0 ** (-np.arange(pairs) / pairs)
    _, got = rnn.kv_append(k, k, kc, kc.clone(), ints([[0]]), ints([0]), ints([0, 3]),
                           inv_freq=torch.from_numpy(inv).cuda(), positions=ints(pos), with_k=True)
    want = oa.rotate(f64(k), np.array(pos)[:, None], inv, False)
    # the angle itself: 2^31 inv in double, off by 2^31 2^-52
    tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * np.abs(f64(k)).max() * 2
    assert np.all(np.abs(f64(got) - want) <= tol)


def test_append_in_place_and_absent_pages():
    g = gen_of(5)
    q, k, v = normal(g, (6, 2, 64), HF), normal(g, (6, 1, 64), HF), normal(g, (6, 1, 64), HF)
    inv = torch.full((32,), 0.25, dtype=torch.float64, device="cuda")
    table = ints([[1, -1], [7, 2]])     # the second page of 0 and the first of 1 do not exist
    kc, vc = (torch.zeros((3, 2, 1, 64), dtype=HF, device="cuda") for _ in range(2))
    want_q, want_k = rnn.kv_append(k, v, kc.clone(), vc.clone(), table, ints([0, 0]),
                                   ints([0, 3, 6]), q=q, inv_freq=inv, with_k=True)
    got_q, got_k = rnn.kv_append(k, v, kc, vc, table, ints([0, 0]), ints([0, 3, 6]), q=q,
                                 inv_freq=inv, q_out=q, k_out=k)
    assert got_q is q and got_k is k
    assert torch.equal(q, want_q) and torch.equal(k, want_k)
    assert torch.equal(kc[1], want_k[:2]) and torch.equal(vc[1], v[:2])
    assert torch.equal(kc[2, 0], want_k[5]) and torch.equal(vc[2, 0], v[5])
    assert (kc[0] == 0).all() and (kc[2, 1] == 0).all()
    # numbers below zero and beyond the table
    kc.zero_()
    rnn.kv_append(k[:2], v[:2], kc, vc, table, ints([-1, 4]), ints([0, 1, 2]))
    assert (kc == 0).all()


# ------------------------------------------------------------ used together
@pytest.mark.parametrize("dtype,hq,hkv,d,size", [(BF, 4, 2, 64, 16), (HF, 3, 3, 96, 7)])
def test_prompt_then_tokens(dtype, hq, hkv, d, size):
    """Prompts go through append and attn_prompt, then three tokens each through append and
    attn_decode; every row equals full causal attention over the rotated tokens."""
    g = gen_of(11)
    first, steps = [37, 130, 1], 3
    B, total = len(first), [n + steps for n in first]
    kc, vc, table = paged(g, total, size, hkv, d, dtype)
    kc.fill_(float("nan"))
    vc.fill_(float("nan"))
    tab = torch.from_numpy(table).cuda()
    inv = torch.from_numpy(10000.0 ** (-np.arange(d // 2) / (d // 2))).cuda()
    q, k, v = (normal(g, (sum(total), h, d), dtype) for h in (hq, hkv, hkv))
    at = cum(total)
    turned_q, turned_k = torch.empty_like(q), torch.empty_like(k)
    prompt = torch.cat([torch.arange(at[b], at[b] + first[b]) for b in range(B)]).cuda()
    qr, kr = rnn.kv_append(k[prompt], v[prompt], kc, vc, tab, ints([0] * B), ints(cum(first)),
                           q=q[prompt], inv_freq=inv, with_k=True)
    out = torch.empty_like(q)
    out[prompt] = rnn.attn_prompt(qr, kr, v[prompt], ints(cum(first)))
    turned_q[prompt], turned_k[prompt] = qr, kr
    lens = ints(first)
    for s in range(steps):
        now = torch.tensor([at[b] + first[b] + s for b in range(B)]).cuda()
        qr, kr = rnn.kv_append(k[now], v[now], kc, vc, tab, lens, ints(list(range(B + 1))),
                               q=q[now], inv_freq=inv, with_k=True)
        lens += 1
        out[now] = rnn.attn_decode(qr, kc, vc, tab, lens)
        turned_q[now], turned_k[now] = qr, kr
    ref = oa.prompt(f64(turned_q), f64(turned_k), f64(v), at, at, True, 1 / math.sqrt(d))
    check_attention(out, None, ref, dtype, d, float(v.abs().max()))


def test_same_bits_again_captured_and_on_another_stream():
    g = gen_of(12)
    q, k, v, cu_q, cu_k, out, lse = run_prompt(BF, [300, 77], [300, 77], 4, 2, 128, True, 12)
    cq, ck = ints(cu_q), ints(cu_k)
    dq, kc, vc, table, dout, dlse = run_decode(BF, [3000, 129], 16, 8, 2, 128, 13)
    tab, lens = torch.from_numpy(table).cuda(), ints([3000, 129])
    inv = torch.full((64,), 0.1, dtype=torch.float64, device="cuda")
    args = (k[:8], v[:8], kc, vc, tab, ints([0, 0]), ints([0, 4, 8]))

    def all_three():
        a = rnn.attn_prompt(q, k, v, cq, ck, with_lse=True)
        b = rnn.attn_decode(dq, kc, vc, tab, lens, with_lse=True)
        return (*a, *b)

    want = (out, lse, dout, dlse)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(all_three(), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = all_three()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = all_three()
        qr, _ = rnn.kv_append(*args, q=q[:8], inv_freq=inv)
    for x in (*got, qr):
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    again, _ = rnn.kv_append(*args, q=q[:8], inv_freq=inv)
    assert torch.equal(qr, again)


def test_decode_row_offsets_beyond_32_bits():
    """A cache of more than 2^32 bytes and 2^31 elements: its last page is read and written."""
    d, hkv, size = 128, 8, 64
    pages = (1 << 31) // (size * hkv * d) + 3
    kc = torch.zeros((pages, size, hkv, d), dtype=BF, device="cuda")
    vc = torch.zeros_like(kc)
    g = gen_of(14)
    k, v = normal(g, (70, hkv, d), BF), normal(g, (70, hkv, d), BF)
    table = ints([[pages - 1, pages - 2]])
    rnn.kv_append(k, v, kc, vc, table, ints([0]), ints([0, 70]))
    assert torch.equal(kc[pages - 1], k[:64]) and torch.equal(vc[pages - 2, :6], v[64:])
    q = normal(g, (1, 16, d), BF)
    out = rnn.attn_decode(q, kc, vc, table, ints([70]))
    ref = oa.prompt(f64(q), f64(k), f64(v), [0, 1], [0, 70], False, 1 / math.sqrt(d))
    check_attention(out, None, ref, BF, d, 6.0)


def test_calls_at_once_on_two_streams():
    g = gen_of(15)
    lens = [1500, 33]
    dq, kc, vc, table, want, want_lse = run_decode(BF, lens, 16, 8, 2, 64, 15)
    tab, lt = torch.from_numpy(table).cuda(), ints(lens)
    q, k, v, cu_q, cu_k, pout, plse = run_prompt(BF, [200, 900], [200, 900], 2, 1, 64, True, 16)
    cq, ck = ints(cu_q), ints(cu_k)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(12):
        with torch.cuda.stream(streams[i % 2]):
            got.append(rnn.attn_decode(dq, kc, vc, tab, lt, with_lse=True) +
                       rnn.attn_prompt(q, k, v, cq, ck, with_lse=True))
    torch.cuda.synchronize()
    for a, al, b, bl in got:
        assert torch.equal(a, want) and torch.equal(al, want_lse)
        assert torch.equal(b, pout) and torch.equal(bl, plse)


FIRST_IN_CAPTURE = """
import torch, reciprocal_nearest_neighbour_b200 as rnn
i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
q = torch.randn(20, 2, 64, device="cuda").bfloat16()
kc = torch.zeros(3, 16, 2, 64, device="cuda").bfloat16()
vc, table, zero, cu, n = kc.clone(), i(2, 0).view(1, 2), i(0), i(0, 20), i(20)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    rnn.kv_append(q, q, kc, vc, table, zero, cu)
    a = rnn.attn_prompt(q, q, q, cu, causal=False)
    b = rnn.attn_decode(q[19:], kc, vc, table, n)
g.replay()
torch.cuda.synchronize()
assert torch.equal(kc[2], q[:16]) and (a[19].float() - b[0].float()).abs().max() < 0.05
"""


def test_first_call_of_a_process_inside_a_capture():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", FIRST_IN_CAPTURE], check=True, timeout=300, cwd=root)
