"""Pins of the 8-bit cache's oracle, by hand and against torch's own e4m3 (CPU)."""
import numpy as np
import pytest
import torch

from oracle import cache_q8 as oq


def test_e4m3_values_are_torchs():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes.copy()).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(oq.e4m3_value(codes), want, equal_nan=True)
    assert oq.e4m3_value(0x7E) == 448 and oq.e4m3_value(0x01) == 2.0 ** -9


def test_nearest_e4m3_is_torchs():
    x = np.concatenate([np.linspace(-448, 448, 4001), np.linspace(-0.05, 0.05, 4001),
                        [17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10]]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    got = oq.nearest_e4m3(x.astype(np.float64))
    assert np.array_equal(got, want)
    assert np.all(np.abs(got - x) <= oq.half_step(x.astype(np.float64), "e4m3"))


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
def test_quantise_by_hand(codes):
    top = oq.TOP[codes]
    x = np.array([[top * 2, -top, 2.0, 0.0], [0.0, 0.0, 0.0, 0.0]])
    v, s = oq.quantise32(x, codes)
    assert s[0] == 2 and s[1] == 2.0 ** -126
    assert np.array_equal(v[0], [top, -top / 2 if codes == "e4m3" else -64, 1, 0])
    assert np.array_equal(v[1], [0, 0, 0, 0])
    assert np.array_equal(oq.scale(x, codes), [2, 2.0 ** -126])
