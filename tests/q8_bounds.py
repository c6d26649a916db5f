"""Error bounds of the 8-bit cache against the double-precision oracle.

u = finfo.eps / 2 of the 16-bit type (bf16 2^-8, fp16 2^-11).

Rotated rows.  The angle's fraction of a turn is rounded to fp32 after it was
doubled (2^-25 of half a turn, 9.4e-8), its cosine and sine have 2 ulp (1.2e-7),
their products with two channels and the sum are fp32 (1.2e-7): together below
2^-21 (|x1| + |x2|), ``turn_error``.  A scale has that relative to the largest channel
and 2^-23 of the quotient.  A held value is off by half a step of its code (at the
largest magnitude that the fp32 row may have) and 3 * 2^-23 for the two quotients and
the product.

Attention, as in attn_bounds.py, of the values code * scale taken as exact:

* u |out| (and 2^-25 below fp16's normal range): the output's own rounding;
* (2^-12 + 2 e + n 2^-23) A, A = sum w|v|: each weight is rounded to fp16 once (half a
  step: 2^-12), has a relative error e = (d + 8) 2^-23 reach + 2^-21 from its score (four
  roundings more than there: the scales and the queries' factor) and its exponential,
  and meets n fp32 additions that cut off;
* n 2^-30 vmax: a weight p vs below fp16's normal range is held to an absolute 2^-25 where
  the largest so far was put at 2^5 or more; relative to it 2^-30 of a value, and no value
  is larger than vmax.

The log-sum has (e + n 2^-23 + |lse| 2^-22 + 2^-20).
"""
import numpy as np
import torch

turn_error = 2.0 ** -21


def check_attention_q8(out, lse, ref, dtype, d, vmax):
    u = torch.finfo(dtype).eps / 2
    got = out.double().cpu().numpy()
    e = (d + 8) * 2.0 ** -23 * ref.reach + 2.0 ** -21
    n = ref.keys
    tol = u * np.abs(ref.out) + (2.0 ** -12 + 2 * e + n * 2.0 ** -23)[..., None] * ref.spread * (1 + 4 * u)
    tol = tol + (n * 2.0 ** -30 * vmax)[..., None]
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25
    err = np.abs(got - ref.out)
    assert np.isfinite(got).all()
    bad = err > tol
    assert not bad.any(), (np.argwhere(bad)[:5], err[bad][:5], tol[bad][:5])
    empty = n == 0
    assert np.all(got[empty] == 0)
    if lse is not None:
        g = lse.double().cpu().numpy()
        assert np.all(np.isneginf(g[empty]))
        full = ~empty
        bound = e + n * 2.0 ** -23 + np.abs(np.where(full, ref.lse, 0)) * 2.0 ** -22 + 2.0 ** -20
        assert np.all(np.abs(g[full] - ref.lse[full]) <= bound[full])
