"""Error bounds of the attention kernels against the double-precision oracle.

Half a step of the 16-bit type is u = finfo.eps / 2 (bf16 2^-8, fp16 2^-11).
An output row is  sum_t p_t v_t / sum_t p_t.  Its error has these parts:

* u |out|: the output's own rounding;
* u A with A = sum w|v| (the weights sum to 1): each p_t is rounded once for
  the second product;
* 2 e A: a relative error e of every weight.  e = (d + 4) 2^-23 reach (fp32
  sums of d exact products and the scaled exponent, reach = scale sum|q k|) +
  2^-21 (exp2 and the final division);
* n 2^-23 A: n fp32 additions of the weighted sum and of the total;
* fp16 only, n 2^-31 max|v|: below fp16's normal range p_t is held to an
  absolute 2^-25, in a row whose largest p is 2^7 or more.  (The kernels scale
  fp16 probabilities by 2^7 or 2^15 at a reference that never exceeds the
  row's maximum.)  And 2^-25 for an output below that range.

The log-sum has (e + n 2^-23 + |lse| 2^-22 + 2^-20).
"""
import numpy as np
import torch


def check_attention(out, lse, ref, dtype, d, vmax):
    u = torch.finfo(dtype).eps / 2
    got = out.double().cpu().numpy()
    e = (d + 4) * 2.0 ** -23 * ref.reach + 2.0 ** -21
    n = ref.keys
    tol = u * np.abs(ref.out) + (u + (2 * e + n * 2.0 ** -23))[..., None] * ref.spread * (1 + 4 * u)
    if dtype == torch.float16:
        tol = tol + (n * 2.0 ** -31 * vmax)[..., None]
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
