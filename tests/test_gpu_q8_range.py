"""attn_decode_q8 over values of any size that the cache holds (needs a B200).

The bounds are those of q8_bounds.py.  They hold at every size: a weight is held to 2^-25
where the head's largest was put at 2^5 or more, whatever the values' scales are.
"""
import math

import numpy as np
import pytest
import torch

import reciprocal_nearest_neighbour_b200 as rnn
from oracle import attention as oa
from oracle import cache_q8 as oq
from q8_bounds import check_attention_q8
from test_gpu_q8 import CODES, deal, f64, filled, gen_of, ints, new_cache, normal, raw

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def check(out, lse, ref, d, vmax):
    """check_attention_q8 for bf16 outputs, of which some lie below 2^-126: bf16's steps are
    2^-133 there, so an output's own rounding is off by up to 2^-134.  (As 2^-12 of the
    weighted |values|, which the bound has.)"""
    ref.spread = ref.spread + 2.0 ** -134 / 2.0 ** -12
    check_attention_q8(out, lse, ref, BF, d, vmax)


def run_decode(codes, lens, hq, hkv, d, size, change, seed=0, std=1.0):
    g = gen_of(seed)
    table, pages = deal(g, lens, size)
    kc, vc, scales, kv, vv = filled(g, codes, pages, size, hkv, d)
    change(table, kc, vc, scales, kv, vv)
    q = normal(g, (len(lens), hq, d), BF, std)
    out, lse = rnn.attn_decode_q8(q, kc, vc, scales, ints(table), ints(lens), with_lse=True)
    check(out, lse, oa.decode(f64(q), kv, vv, table, lens, 1 / math.sqrt(d)), d, np.abs(vv).max())


def shrink(scales, vv, factor):
    """The values' scales times `factor` (per row, or one), but no smaller than an append's."""
    old = scales[..., 1].cpu().double()
    new = (old * torch.as_tensor(factor)).clamp_min(2.0 ** -126).float()
    scales[..., 1] = new.cuda()
    vv *= (new.double() / old).numpy().transpose(0, 2, 1)[..., None]


def all_by(power):
    return lambda table, kc, vc, scales, kv, vv: shrink(scales, vv, 2.0 ** power)


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
@pytest.mark.parametrize("power", [-40, -54, -70, -90, -110, -118, 40, 90])
@pytest.mark.parametrize("d", [64, 128])
def test_values_of_one_size(codes, power, d):
    run_decode(codes, [70, 133, 1, 515], 4, 2, d, 16, all_by(power), seed=d)
    run_decode(codes, [45, 300], 20, 2, d, 24, all_by(power), seed=d, std=3.0)


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
@pytest.mark.parametrize("power", [-70, -90, -118])
def test_small_values_over_many_blocks(codes, power):
    """Pairs that several CTAs share, and CTAs with several pairs."""
    run_decode(codes, [3000, 9, 5000], 4, 2, 64, 16, all_by(power))
    run_decode(codes, [1280] * 40, 4, 4, 128, 16, all_by(power))


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
@pytest.mark.parametrize("up", [True, False])
@pytest.mark.parametrize("lens", [[900], [9000, 40]])
def test_sizes_that_rise_or_fall_along_a_sequence(codes, up, lens):
    """Over 116 powers of two, from the smallest or to it."""
    def change(table, kc, vc, scales, kv, vv):
        f = torch.ones(scales.shape[:3], dtype=torch.float64)
        for b, n in enumerate(lens):
            for t in range(n):
                at = t / n if up else 1 - t / n
                f[table[b, t // 16], :, t % 16] = 2.0 ** (116 * (at - 1))
        shrink(scales, vv, f)

    run_decode(codes, lens, 3, 1, 64, 16, change)


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
@pytest.mark.parametrize("apart", [40, 80, 118])
@pytest.mark.parametrize("heavy_first", [True, False])
def test_small_values_of_heavy_keys_beside_large_ones_of_light_keys(codes, apart, heavy_first):
    """Keys of score 0 with values 2^-apart, and of score -apart log 2 with values of 1: the
    two meet in the sum at one size."""
    g, n, size, d = gen_of(apart), 500, 16, 64
    table, pages = deal(g, [n], size)
    kc, vc, scales, kv, vv = filled(g, codes, pages, size, 1, d, spread=0.0)
    heavy = np.arange(n) < n // 2 if heavy_first else np.arange(n) >= n // 2
    page, row = table[0, np.arange(n) // size], np.arange(n) % size
    low = np.float32(apart * np.log(2) / 96)
    kc.view(torch.uint8).zero_()                       # a zero in either type
    code = torch.tensor([-96.0]).to(CODES[codes]).view(torch.uint8).item()
    light = ints(page[~heavy]).long(), ints(row[~heavy]).long()
    kc.view(torch.uint8)[light[0], light[1], 0, 0] = code
    scales[..., 0] = float(low)
    kv[:] = 0
    kv[page[~heavy], row[~heavy], 0, 0] = -96 * float(low)
    f = torch.ones(scales.shape[:3], dtype=torch.float64)
    f[page[heavy], 0, row[heavy]] = 2.0 ** -apart
    shrink(scales, vv, f)
    q = torch.zeros(1, 2, d, dtype=BF, device="cuda")
    q[..., 0] = torch.tensor([1.0, 0.5], device="cuda")
    out, lse = rnn.attn_decode_q8(q, kc, vc, scales, ints(table), ints([n]), scale=1.0, with_lse=True)
    ref = oa.decode(f64(q), kv, vv, table, [n], 1.0)
    # the largest weighted value takes the place of the largest value: no weight is put above it
    w = np.exp(np.einsum("hc,kc->hk", f64(q[0]), kv[page, row, 0]) - ref.lse[0][:, None])
    most = (w * np.abs(vv[page, row, 0]).max(-1)).max(-1)
    for h in range(2):
        one = oa.Attn(*(x[:, h:h + 1] for x in (ref.out, ref.lse, ref.spread, ref.reach, ref.keys)))
        check(out[:, h:h + 1], lse[:, h:h + 1], one, d, most[h])


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
@pytest.mark.parametrize("size", [1e-20, 1e-27, 1e-33, 1e-36, 1e30])
def test_append_decode_and_read_back_agree(codes, size):
    """bf16 values of one size: what is attended to is what is read back."""
    g, n, d = gen_of(3), 300, 64
    table, pages = deal(g, [n], 16)
    kc, vc, scales = new_cache(codes, pages, 16, 2, d)
    q, k = normal(g, (1, 4, d), BF), normal(g, (n, 2, d), BF)
    v = (torch.randn(n, 2, d, generator=g).double() * size).to(BF).cuda()
    rnn.kv_append_q8(k, v, kc, vc, scales, ints(table), ints([0]), ints([0, n]))
    kr, vr = rnn.kv_read_q8(kc, vc, scales, ints(table), ints([0, n]), n, BF)
    out, lse = rnn.attn_decode_q8(q, kc, vc, scales, ints(table), ints([n]), with_lse=True)
    values = [oq.value(raw(c), codes) * f64(scales)[..., w].transpose(0, 2, 1)[..., None]
              for w, c in enumerate((kc, vc))]
    ref = oa.decode(f64(q), *values, table, [n], d ** -0.5)
    check(out, lse, ref, d, float(vr.double().abs().max()) * (1 + 2.0 ** -8))
    page, row = table[0, np.arange(n) // 16], np.arange(n) % 16
    want = values[1][page, row]
    # read back: the product with the scale and bf16's own rounding, of normal numbers
    assert np.all(np.abs(f64(vr) - want) <= 1.01 * 2.0 ** -8 * np.abs(want) + 2.0 ** -133)


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
@pytest.mark.parametrize("d", [64, 128])
def test_scales_of_zero_and_rows_without_size(codes, d):
    """Values of scale 0 weigh nothing, wherever they stand, and do not hide small ones."""
    def change(table, kc, vc, scales, kv, vv):
        f = torch.full(scales.shape[:3], 2.0 ** -100, dtype=torch.float64)
        shrink(scales, vv, f)
        for b, rows in ((0, range(0, 200)), (1, range(100, 133))):
            for t in rows:
                pg, r = table[b, t // 16], t % 16
                scales[pg, :, r, 1] = 0
                vv[pg, r] = 0

    run_decode(codes, [515, 133], 4, 2, d, 16, change)
