"""A plain float64 attention row with a derived bound on a kernel's error
(test infrastructure)."""

from __future__ import annotations

import numpy as np

HALF_BF16 = 2.0 ** -8   # half a step of bf16, relative to the value
EPS32 = 2.0 ** -24


def attend_row(q, K, V, gate=None):
    """q [Hq, D]; K, V [n, Hkv, D] of the tokens the row sees; gate [Hq, D] or
    None.  Returns (out, bound), both [Hq, D], unrounded.

    The bound, with w the softmax weights, o = sum w v, A = sum w |v|:
      scores   fp32 sums of exact products: D * 2^-24 * sum |q k| / sqrt(D),
               and 2^-22 |s| for the base-2 exponential's argument; a score off
               by d moves every weight by at most e^(2d) - 1, o by that times A;
      weights  rounded to bf16 or f16 before the product: 2^-8 A;
               f16 weights below its normal range, relative to a reference
               that a weight may pass by 2^8: n * 2^-25 * max |v|;
      sums     fp32 over n tokens, the exponential's own error: (n + 64) * 2^-24 A;
      output   rounded to bf16: 2^-8 |o|; after the gate once more."""
    Hq, D = q.shape
    n, Hkv = K.shape[0], K.shape[1]
    out, bound = np.zeros((Hq, D)), np.zeros((Hq, D))
    if n:
        G = Hq // Hkv
        for h in range(Hq):
            k, v = K[:, h // G], V[:, h // G]
            z = (k @ q[h]) / np.sqrt(D)
            d = (D * EPS32 * (np.abs(k) @ np.abs(q[h])) / np.sqrt(D)).max() + 4 * EPS32 * np.abs(z).max()
            w = np.exp(z - z.max())
            w /= w.sum()
            o, A = w @ v, w @ np.abs(v)
            out[h] = o
            bound[h] = (A * (np.expm1(2 * d) + HALF_BF16 + (n + 64) * EPS32) + n * 2.0 ** -25 * w.max() * np.abs(v).max()
                        + HALF_BF16 * np.abs(o))
            bound[h] *= 1 + 2 * HALF_BF16
    if gate is not None:
        s = 1.0 / (1.0 + np.exp(-gate))
        out, bound = out * s, bound * s * (1 + 2.0 ** -20) + (HALF_BF16 + 2.0 ** -20) * np.abs(out * s)
        bound *= 1 + 2 * HALF_BF16
    return out, bound + 1e-30


def assert_row(got, q, K, V, gate=None, what=""):
    want, bound = attend_row(q, K, V, gate)
    off = np.abs(got - want)
    worst = float((off / bound).max())
    assert np.isfinite(got).all() and worst <= 1.0, f"{what}: {worst:.2f} of the bound, off by {off.max():.3g}"
