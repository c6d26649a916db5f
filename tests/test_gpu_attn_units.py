"""attn_prompt beyond one unit a CTA (more units than SMs, units of very different
length, waits that last a whole unit, rows longer than one accumulator holds, units that
are given up), and attn_decode with large groups of heads and long rows."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import reciprocal_nearest_neighbour_b200 as rnn
from attn_bounds import check_attention
from oracle.attention import Attn

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cum(lens):
    return [0] + np.cumsum(lens).tolist()


def normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


def reference(q, k, v, cu_q, cu_k, causal, scale) -> Attn:
    """Attention in 64 bits, a sequence at a time, with what the error bounds need."""
    tq, hq, d = q.shape
    group = hq // k.shape[1]
    opt = dict(dtype=torch.float64, device="cuda")
    out, spread = torch.zeros(q.shape, **opt), torch.zeros(q.shape, **opt)
    lse, reach = torch.full((tq, hq), -math.inf, **opt), torch.zeros((tq, hq), **opt)
    keys = torch.zeros((tq, hq), dtype=torch.int64, device="cuda")
    for b in range(len(cu_q) - 1):
        nq, nk = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        if nq == 0 or nk == 0:
            continue
        seen = torch.arange(nq, device="cuda") + (nk - nq + 1) if causal else \
            torch.full((nq,), nk, device="cuda")
        seen = seen.clamp(0, nk)
        hidden = torch.arange(nk, device="cuda")[None] >= seen[:, None]
        some = seen > 0
        for h in range(hq):
            K = k[cu_k[b]:cu_k[b + 1], h // group].double()
            V = v[cu_k[b]:cu_k[b + 1], h // group].double()
            Q = q[cu_q[b]:cu_q[b + 1], h].double()
            s = ((Q @ K.T) * scale).masked_fill(hidden, -math.inf)
            top = s.amax(1, keepdim=True).masked_fill(~some[:, None], 0.0)
            w = (s - top).exp()
            total = w.sum(1, keepdim=True)
            one = torch.where(some[:, None], total, 1.0)
            at = slice(cu_q[b], cu_q[b + 1])
            out[at, h], spread[at, h] = (w @ V) / one, (w @ V.abs()) / one
            lse[at, h] = torch.where(some, (top + one.log())[:, 0], -math.inf)
            reach[at, h] = ((Q.abs() @ K.abs().T) * scale).masked_fill(hidden, 0.0).amax(1)
            keys[at, h] = seen
    return Attn(*(x.cpu().numpy() for x in (out, lse, spread, reach, keys)))


def ragged(seed):
    """72 sequences (three groups of 32 as the kernel deals them): long ones between ones
    without keys, without queries, and with rows or whole tiles that see nothing."""
    rng = np.random.default_rng(seed)
    nq, nk = [], []
    for b in range(72):
        kind = b % 9
        n = int(rng.integers(1, 420))
        if kind < 4:                       # as many keys as queries, or more
            nq.append(n)
            nk.append(n + int(rng.integers(0, 500)) * (kind & 1))
        elif kind == 4:                    # the first 128 rows see nothing, the next do
            nq.append(200 + n % 50)
            nk.append(60 + n % 30)
        elif kind == 5:                    # only the last rows of several tiles see a key
            nq.append(n + 300)
            nk.append(1 + n % 20)
        elif kind == 6:                    # many key tiles for a few queries
            nq.append(1 + n % 9)
            nk.append(900 + 2 * n)
        elif kind == 7:
            nq.append(n)
            nk.append(0)
        else:
            nq.append(0)
            nk.append(n)
    return nq, nk


def inputs(dtype, nq, nk, hq, hkv, d, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    q, k, v = (normal(g, (sum(n), h, d), dtype) for n, h in ((nq, hq), (nk, hkv), (nk, hkv)))
    return q, k, v, cum(nq), cum(nk)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (6, 2)])     # pairs of heads, pairs of token tiles
@pytest.mark.parametrize("causal", [True, False])
def test_many_ragged_units(dtype, d, hq, hkv, causal):
    q, k, v, cu_q, cu_k = inputs(dtype, *ragged(d + hq), hq, hkv, d, 21)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    args = (q, k, v, ints(cu_q), ints(cu_k))
    out, lse = rnn.attn_prompt(*args, causal=causal, with_lse=True, workspace=ws)
    rnn.workspace_status(ws)
    ref = reference(q, k, v, cu_q, cu_k, causal, 1 / math.sqrt(d))
    check_attention(out, lse, ref, dtype, d, float(v.abs().max()))
    for _ in range(3):                    # units are dealt as CTAs come free, results are not
        again, lse2 = rnn.attn_prompt(*args, causal=causal, with_lse=True)
        assert torch.equal(again, out) and torch.equal(lse2, lse)


@pytest.mark.parametrize("d", [40, 64, 96, 128])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (9, 3)])
def test_many_units_of_one_sequence(d, hq, hkv):
    """More units than SMs, up to 41 key tiles each, and more keys than queries."""
    nq, nk = [5003], [5201]
    q, k, v, cu_q, cu_k = inputs(BF, nq, nk, hq, hkv, d, 22)
    for causal in (True, False):
        out, lse = rnn.attn_prompt(q, k, v, ints(cu_q), ints(cu_k), causal=causal, with_lse=True)
        ref = reference(q, k, v, cu_q, cu_k, causal, 1 / math.sqrt(d))
        check_attention(out, lse, ref, BF, d, float(v.abs().max()))


# ---------------------------------------------------- decode forms of large groups
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(9, 1), (16, 1), (34, 2), (40, 1)])
@pytest.mark.parametrize("lens", [[130, 0, 5, 64], [3777, 20]])  # in one share, and joined
def test_decode_groups(dtype, d, hq, hkv, lens):
    """More than 8 query heads a key head, and more than the 16 of one unit."""
    g = torch.Generator("cuda").manual_seed(hq + d)
    size = 48
    need = [-(-n // size) for n in lens]
    deal = torch.randperm(sum(need) + 1, generator=g, device="cuda").int()
    table = torch.zeros((len(lens), max(need)), dtype=torch.int32, device="cuda")
    kc, vc = (normal(g, (sum(need) + 1, size, hkv, d), dtype) for _ in range(2))
    at, rows = 0, []
    for b, n in enumerate(need):
        table[b, :n] = deal[at:at + n]
        rows.append(deal[at:at + n].long())
        at += n
    q = normal(g, (len(lens), hq, d), dtype)
    out, lse = rnn.attn_decode(q, kc, vc, table, ints(lens), with_lse=True)
    k, v = (torch.cat([c[r].flatten(0, 1)[:n] for r, n in zip(rows, lens)]) for c in (kc, vc))
    ref = reference(q, k, v, list(range(len(lens) + 1)), cum(lens), False, 1 / math.sqrt(d))
    check_attention(out, lse, ref, dtype, d, float(v.abs().max()))


# ------------------------------------------------------------------ long waits
def test_unit_longer_than_the_wait_limit():
    """One query over 250 million keys: a single unit of two million steps, well over the
    second after which a wait gives up."""
    n = 250_000_037
    kv = torch.ones((n, 1, 8), dtype=BF, device="cuda")
    q = torch.zeros((1, 1, 8), dtype=BF, device="cuda")
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    out, lse = rnn.attn_prompt(q, kv, kv, ints([0, 1]), ints([0, n]), causal=False, with_lse=True,
                               workspace=ws)
    rnn.workspace_status(ws)
    assert out.isfinite().all()
    # equal scores: the total, n below 2^28 in steps of 128, rounds in its last addition only
    assert abs(float(lse) - math.log(n)) <= math.log(n) * 2.0 ** -22 + 2.0 ** -20


def test_search_longer_than_the_wait_limit():
    """13 million sequences of which the last has rows: the search for its unit, and past the
    blocks of the others, lasts longer than a wait may without anything done."""
    B, n = 13_000_000, 130
    g = torch.Generator("cuda").manual_seed(31)
    q, k, v = (normal(g, (n, h, 64), BF) for h in (2, 1, 1))
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    cu[-1] = n
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    out = rnn.attn_prompt(q, k, v, cu, workspace=ws)
    rnn.workspace_status(ws)
    assert torch.equal(out, rnn.attn_prompt(q, k, v, ints([0, n])))


# ------------------------------------------------------------------- long sums
def held(ref, segment):
    """The oracle's results with the number of keys that meet in one accumulator: `segment`
    of them, then one addition for each of the segments."""
    ref.keys = np.minimum(ref.keys, segment) + ref.keys // segment
    return ref


def test_sum_of_many_equal_weights():
    """250 million equal scores.  Values that are powers of two make every partial sum of up
    to 65536 of them exact; the other additions are rounded to nearest."""
    n = 250_000_037
    values = torch.tensor([2.0 ** (c - 4) for c in range(8)], device="cuda").to(BF)
    kv = torch.empty((n, 1, 8), dtype=BF, device="cuda")
    kv[:] = values
    q = torch.zeros((1, 1, 8), dtype=BF, device="cuda")
    out = rnn.attn_prompt(q, kv, kv, ints([0, 1]), ints([0, n]), causal=False)
    # 3815 additions of a power of two (exact below 2^24 of them) and the ragged end
    assert torch.equal(out[0, 0], values)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d", [40, 64, 96, 128])
@pytest.mark.parametrize("hq", [2, 3])
def test_prompt_long_sums(dtype, d, hq):
    """Values of one sign: what an accumulator loses shows in every channel.  Beside the
    long sequence short ones, and one whose scores grow and fall over its length, so that
    parts taken out early and late count."""
    g = torch.Generator("cuda").manual_seed(d)
    nq, nk = [3, 40, 150, 2], [1 << 22, 40, 70_001, 65_537]
    cu_q, cu_k = cum(nq), cum(nk)
    q = normal(g, (sum(nq), hq, d), dtype) * 0.5
    k = normal(g, (sum(nk), 1, d), dtype)
    v = torch.rand((sum(nk), 1, d), generator=g, device="cuda").add(0.5).to(dtype)
    q[cu_q[2]:cu_q[3], :, 0] = math.sqrt(d)         # scaled scores from -8 to 8
    k[cu_k[2]:cu_k[3], 0, 0] = (torch.linspace(0, 2 * math.pi, nk[2], device="cuda").sin()
                                * 8).to(dtype)
    for causal in (False, True):
        ws = torch.empty(256, dtype=torch.uint8, device="cuda")
        out, lse = rnn.attn_prompt(q, k, v, ints(cu_q), ints(cu_k), causal=causal, with_lse=True,
                                   workspace=ws)
        rnn.workspace_status(ws)
        ref = held(reference(q, k, v, cu_q, cu_k, causal, 1 / math.sqrt(d)), 65536)
        check_attention(out, lse, ref, dtype, d, 1.5)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d,hq", [(8, 3), (72, 3), (8, 10), (72, 10)])
def test_decode_long_sums(dtype, d, hq):
    """300 sequences on the same pages, so that a warp takes four million keys of one of
    them; values of one sign, equal scores, and scores that grow and fall."""
    g = torch.Generator("cuda").manual_seed(d)
    n, size, B = (1 << 24) + 70_001, 64, 300
    pages = -(-n // size)
    k, v = (torch.zeros((pages, size, 1, d), dtype=dtype, device="cuda") for _ in range(2))
    k.normal_(generator=g)
    v.uniform_(0.5, 1.5, generator=g)
    q = normal(g, (3, hq, d), dtype) * 0.5
    q[1:, :, 0] = math.sqrt(d)                          # scaled scores of -8 to 8
    q[0] = 0
    k.view(-1, d)[:, 0] = (torch.linspace(0, 6 * math.pi, pages * size, device="cuda").sin()
                           * 8).to(dtype)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").expand(B, -1)
    kind = [0, 1, 2] * (B // 3)
    lens = [(n, n, 70_001)[x] for x in kind]
    out, lse = rnn.attn_decode(q[kind], k, v, table, ints(lens), with_lse=True)
    for r, many in enumerate((n, n, 70_001)):
        ref = held(reference(q[r:r + 1], k.view(-1, 1, d), v.view(-1, 1, d), [0, 1], [0, many],
                             False, 1 / math.sqrt(d)), 65536)
        for b in (r, 150 + r, B - 3 + r):
            check_attention(out[b:b + 1], lse[b:b + 1], ref, dtype, d, 1.5)


LONG_FIRST_IN_CAPTURE = """
import torch, reciprocal_nearest_neighbour_b200 as rnn
i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
n = 300000
q = torch.randn(4, 2, 64, device="cuda").bfloat16()
kc = torch.randn(n // 64 + 1, 64, 2, 64, device="cuda").bfloat16()
kv = kc.view(-1, 2, 64)[:n]
table = torch.arange(kc.shape[0], dtype=torch.int32, device="cuda").view(1, -1)
cu, ck, lens, one = i(0, 4), i(0, n), i(n), i(n)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    a = rnn.attn_prompt(q, kv, kv, cu, ck, causal=False)
    b = rnn.attn_decode(q[3:], kc, kc, table, lens)
for x in (a, b):
    x.fill_(7)
g.replay()
torch.cuda.synchronize()
s = torch.einsum("hc,khc->hk", q[3].double(), kv.double()) / 8
want = torch.einsum("hk,khc->hc", s.softmax(1), kv.double())
for x in (a[3], b[0]):
    assert (x.double() - want).abs().max() < 2e-2
"""


def test_first_long_call_of_a_process_inside_a_capture():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", LONG_FIRST_IN_CAPTURE], check=True, timeout=300, cwd=root)


# --------------------------------------------------------------- units given up
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (6, 2)])
@pytest.mark.parametrize("on", [1, 2])
@pytest.mark.parametrize("many", [False, True])
def test_rows_given_up_are_nan(d, hq, hkv, on, many):
    """A wait that runs out leaves no old bytes in the rows, with or without a workspace; units
    that a CTA had finished before keep their results.  With many keys in the call too."""
    nq, nk = ragged(5)
    nk = [max(1, n) for n in nk]
    if many:
        nq, nk = nq + [130], nk + [70_001]
    q, k, v, cu_q, cu_k = inputs(BF, nq, nk, hq, hkv, d, 23)
    front = torch.full((3, hq, d), 7.0, dtype=BF, device="cuda")
    args = (torch.cat([front, q]), k, v, ints([3 + x for x in cu_q]), ints(cu_k))
    want, want_lse = rnn.attn_prompt(*args, causal=False, with_lse=True)
    out = torch.full_like(want, 7.0)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    lib = rnn._lib.load()
    lib.rnn_test_stall_loads(on, 20_000_000)
    try:
        _, lse = rnn.attn_prompt(*args, causal=False, with_lse=True, out=out, workspace=ws)
        bare = rnn.attn_prompt(*args, causal=False)
        torch.cuda.synchronize()
    finally:
        lib.rnn_test_stall_loads(0, 0)
    with pytest.raises(rnn.RNNError):
        rnn.workspace_status(ws)
    assert (out[:3] == 7).all()
    gone = out[3:].isnan()
    assert torch.equal(gone.all(2), gone.any(2)) and torch.equal(gone.any(2), lse[3:].isnan())
    assert gone.all() if on == 1 else 0.2 < gone.float().mean() < 0.8
    assert torch.equal(out[3:][~gone], want[3:][~gone])
    kept = ~gone.any(2)
    assert torch.equal(lse[3:][kept], want_lse[3:][kept])
    gone = bare[3:].isnan()
    assert gone.any() and torch.equal(bare[3:][~gone], want[3:][~gone])
    again = rnn.attn_prompt(*args, causal=False, workspace=ws)
    rnn.workspace_status(ws)
    assert torch.equal(again[3:], want[3:])


# --------------------------------------------------------------- scores of any size
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size,scale", [(1.0, 1e38), (-1.0, 1e38), (1.0, 2.0 ** 30), (-1.0, 2e6)])
def test_scores_of_any_size(dtype, d, size, scale):
    """Scaled scores up to and beyond fp32's range, of either sign: equal ones weigh the same,
    the others nothing.  All products are exact: keys of 8 and 16, and one of zeros."""
    n = 300
    q = torch.full((n, 2, d), size, dtype=dtype, device="cuda")
    q[:, 1] = 0                                  # scores of 0 beside them
    k = torch.full((n, 1, d), 8.0, dtype=dtype, device="cuda")
    k[1::2] *= 2                                 # every second key
    v = torch.ones((n, 1, d), dtype=dtype, device="cuda")
    v[1::2] = 3
    many = torch.arange(1, n + 1, device="cuda").float()
    odd = (many / 2).floor()                     # keys of 16 among those seen
    best = torch.where(odd > 0, 3.0, 1.0) if size > 0 else torch.ones_like(many)
    want = best[:, None].expand(n, d)
    out, lse = rnn.attn_prompt(q, k, v, ints([0, n]), scale=scale, with_lse=True)
    assert torch.equal(out[:, 0].float(), want)
    mean = (many + 2 * odd) / many
    u = torch.finfo(dtype).eps / 2
    assert ((out[:, 1, 0].float() - mean).abs() <= u * mean * (1 + 2.0 ** -8)).all()
    top = (8.0 * d * size * torch.where(odd > 0, 2.0, 1.0) if size > 0 else
           torch.full_like(many, 8.0 * d * size)).double() * float(torch.tensor(scale))
    count = torch.where(odd > 0, odd, many) if size > 0 else many - odd
    ref = top + count.double().log()
    far = top.abs() > 3.4e38
    assert torch.equal(lse[far, 0].double(), torch.sign(top[far]) * math.inf)
    assert ((lse[:, 0] - ref).abs()[~far] <= ref.abs()[~far] * 2.0 ** -22 + 2.0 ** -20).all()
    assert (lse[:, 1] - many.log()).abs().max() < 1e-5
    cache = [torch.nn.functional.pad(x, (0, 0, 0, 0, 0, 20)).view(20, 16, 1, d) for x in (k, v)]
    table = torch.arange(20, dtype=torch.int32, device="cuda").expand(2, -1)
    dec, dlse = rnn.attn_decode(q[:2], *cache, table, ints([n, 3]), scale=scale, with_lse=True)
    for b, r in ((0, n - 1), (1, 2)):
        assert torch.equal(dec[b, 0], out[r, 0])
        assert abs(float(dec[b, 1, 0]) - float(mean[r])) <= u * float(mean[r]) * (1 + 2.0 ** -8)
        assert torch.equal(dlse[b, 0], lse[r, 0]) or \
            abs(float(dlse[b, 0] - lse[r, 0])) <= float(ref[r].abs()) * 2.0 ** -22 + 2.0 ** -20


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d", [64, 128])
def test_large_scores_growing(dtype, d):
    """Scores of a hundred million that grow key by key: each row takes its last key."""
    n = 500
    q = torch.full((n, 1, d), 64.0, dtype=dtype, device="cuda")
    k = (torch.arange(n, device="cuda").float() / 4).floor()[:, None, None].expand(n, 1, d)
    k = (k * 2).to(dtype).contiguous()           # steps of 2 up to 248: exact in both types
    v = torch.randn((n, 1, d), device="cuda").to(dtype)
    out = rnn.attn_prompt(q, k, v, ints([0, n]), scale=64.0)
    i = torch.arange(n, device="cuda")
    first = i // 4 * 4
    sums = torch.stack([v[first[r]:r + 1, 0].double().mean(0) for r in range(n)])
    u = torch.finfo(dtype).eps / 2
    # up to four equal weights, each exactly 1: the output's rounding and a few fp32 ones
    assert ((out[:, 0].double() - sums).abs() <= sums.abs() * u * (1 + u) + 2.0 ** -20).all()
