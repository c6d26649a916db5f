"""Sums over more keys than one accumulator takes (needs a B200): attn_decode_q8 and both
parts of attn_decode_shared, where a warp or a row tile really has that many keys."""
import math

import numpy as np
import pytest
import torch

import reciprocal_nearest_neighbour_b200 as rnn
from attn_bounds import check_attention
from q8_bounds import check_attention_q8
from test_gpu_attn_units import held, normal, reference

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
HOLD = 65536                       # keys that meet in one accumulator


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def wave(n, turns):
    """Scaled scores that grow and fall, -8 to 8."""
    return torch.linspace(0, 2 * turns * math.pi, n, device="cuda").sin() * 8


@pytest.mark.parametrize("codes", [torch.float8_e4m3fn, torch.int8])
@pytest.mark.parametrize("d,hq", [(8, 3), (72, 3), (8, 10), (72, 10)])
@pytest.mark.parametrize("small", [False, True])
def test_decode_q8(codes, d, hq, small):
    """300 sequences on the same pages over 444 CTAs or fewer: a share is two thirds of one
    and more, so that a warp takes millions of its keys.  Values of one sign; equal scores,
    and scores that grow and fall; scales of about 1, and of 2^-100."""
    g = torch.Generator("cuda").manual_seed(d)
    n, size, B = (1 << 24) + 70_001, 64, 300
    pages = -(-n // size)
    rows = pages * size
    # -(-n // 128) tiles of 128 keys a sequence, B of them over at most 3 * 148 CTAs, 32 keys
    # a warp and tile
    assert B * (n // 128) // 444 * 32 > 16 * HOLD
    ks, vs = (1 / 15, 1 / 80) if codes == torch.int8 else (1 / 32, 1.0)
    k = torch.randn((rows, d), generator=g, device="cuda")
    k[:, 0] = wave(rows, 3)
    k = (k / ks).round_().clamp_(-120, 120) if codes == torch.int8 else k / ks
    kc = k.to(codes)
    del k
    v = torch.empty((rows, d), device="cuda").uniform_(0.5, 1.5, generator=g)
    vc = ((v / vs).round_() if codes == torch.int8 else v).to(codes)
    del v
    scales = torch.empty((pages, 1, size, 2), device="cuda")
    scales[..., 0] = ks
    scales[..., 1].uniform_(0.5, 1.0, generator=g)
    scales[..., 1] *= vs * (2.0 ** -100 if small else 1.0)
    q = normal(g, (3, hq, d), BF) * 0.5
    q[1:, :, 0] = math.sqrt(d)
    q[0] = 0
    table = torch.arange(pages, dtype=torch.int32, device="cuda").expand(B, -1)
    kind = [0, 1, 2] * (B // 3)
    many = (n, n, 70_001)
    out, lse = rnn.attn_decode_q8(q[kind], kc.view(pages, size, 1, d), vc.view(pages, size, 1, d),
                                  scales, table, ints([many[x] for x in kind]), with_lse=True)
    k64 = kc.double() * scales[..., 0].reshape(-1, 1).double()
    v64 = vc.double() * scales[..., 1].reshape(-1, 1).double()
    del kc, vc
    top = float(v64.max())
    for r in range(3):
        ref = held(reference(q[r:r + 1], k64[:, None], v64[:, None], [0, 1], [0, many[r]], False,
                             1 / math.sqrt(d)), HOLD)
        for b in (r, 150 + r, B - 3 + r):
            check_attention_q8(out[b:b + 1], lse[b:b + 1], ref, BF, d, top)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d,hq", [(8, 3), (72, 3), (8, 10), (72, 10)])
def test_shared_own_rows(dtype, d, hq):
    """The sequences' own rows: 300 on the same pages behind a prefix."""
    g = torch.Generator("cuda").manual_seed(d)
    n, size, B, ahead = (1 << 24) + 70_001, 64, 300, 1000
    pages = -(-n // size)
    assert B * (n // 128) // 296 * 16 > 16 * HOLD
    k, v = (torch.zeros((pages, size, 1, d), dtype=dtype, device="cuda") for _ in range(2))
    k.normal_(generator=g)
    v.uniform_(0.5, 1.5, generator=g)
    k.view(-1, d)[:, 0] = wave(pages * size, 3).to(dtype)
    q = normal(g, (3, hq, d), dtype) * 0.5
    q[1:, :, 0] = math.sqrt(d)
    q[0] = 0
    table = torch.arange(pages, dtype=torch.int32, device="cuda").expand(B, -1)
    first = pages // 2                       # the prefix's pages, some of those in the middle
    names = torch.arange(first, first + -(-ahead // size), dtype=torch.int32, device="cuda")
    kind = [0, 1, 2] * (B // 3)
    many = (n, n, 70_001)
    out, lse = rnn.attn_decode_shared(q[kind], k, v, names, ints([ahead]), table,
                                      ints([many[x] for x in kind]), with_lse=True)
    kf, vf = k.view(-1, 1, d), v.view(-1, 1, d)
    pre = slice(first * size, first * size + ahead)
    for r in range(3):
        kk, vv = (torch.cat([x[pre], x[:many[r]]]) for x in (kf, vf))
        ref = held(reference(q[r:r + 1], kk, vv, [0, 1], [0, len(kk)], False, 1 / math.sqrt(d)), HOLD)
        for b in (r, 150 + r, B - 3 + r):
            check_attention(out[b:b + 1], lse[b:b + 1], ref, dtype, d, 1.5)


def blocks(B, hq, hkv, d, room):
    """CTAs that the prefix is cut over: each has a part of 256 rows in the workspace."""
    size = rnn._lib.load().rnn_attn_decode_shared_workspace_size
    whole = hkv * -(-B * (hq // hkv) // 256)             # one key tile: a CTA a unit
    a_part = 2 * 128 * ((64 if d <= 64 else 128) * 4 + 8)
    more, rest = divmod(size(B, hq, hkv, d, room) - size(B, hq, hkv, d, 1), a_part)
    assert rest == 0
    return whole, whole + more


# units of 256 rows (wide), the same with a last one of 128 (narrow), and many key heads with
# up to 128 rows each (narrow only)
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("B,hq,hkv", [(2368, 16, 2), (2320, 16, 2), (100, 148, 148)])
@pytest.mark.parametrize("d", [40, 128])
def test_shared_prefix(dtype, B, hq, hkv, d):
    """More key heads and rows than CTAs run at once: no plan cuts the prefix finer than its
    accumulators have to be, 64000 keys each (32000 in the two of a narrow unit)."""
    g = torch.Generator("cuda").manual_seed(B)
    prefix = 4 * HOLD - 3000
    whole, ctas = blocks(B, hq, hkv, d, prefix)
    assert ctas <= 4 * whole
    size, pages = 64, 512                                # 32768 rows, again and again
    k, v = (torch.zeros((pages + 1, size, hkv, d), dtype=dtype, device="cuda") for _ in range(2))
    k.normal_(generator=g)
    v.uniform_(0.5, 1.5, generator=g)
    k.view(-1, hkv, d)[:, :, 0] = wave((pages + 1) * size, 2).to(dtype)[:, None]
    q = normal(g, (B, hq, d), dtype) * 0.5
    q[1::2, :, 0] = math.sqrt(d)
    q[::2] = 0
    names = torch.arange(-(-prefix // size), dtype=torch.int32, device="cuda") % pages
    table = torch.full((B, 1), pages, dtype=torch.int32, device="cuda")
    lens = [(7 * b) % 50 for b in range(B)]
    out, lse = rnn.attn_decode_shared(q, k, v, names, ints([prefix]), table, ints(lens), with_lse=True)
    at = torch.arange(prefix, device="cuda") % (pages * size)
    kf, vf = k.view(-1, hkv, d), v.view(-1, hkv, d)
    for b in (0, 1, B // 2, B - 1):
        for h in sorted({0, hq // 2, hq - 1}):
            hk = h // (hq // hkv)
            kk, vv = (torch.cat([x[at, hk], x[pages * size:][:lens[b], hk]])[:, None] for x in (kf, vf))
            ref = held(reference(q[b:b + 1, h:h + 1], kk, vv, [0, 1], [0, len(kk)], False,
                                 1 / math.sqrt(d)), HOLD)
            check_attention(out[b:b + 1, h:h + 1], lse[b:b + 1, h:h + 1], ref, dtype, d, 1.5)
