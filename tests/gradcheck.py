"""Tolerances of the gradients against the fp64 oracle.

A gradient is a sum of terms computed in fp32 and rounded once to its type:
  |got - ref| <= half a step of the type at ref + K 2^-24 mag,
with mag the sum of the terms' magnitudes (oracle/backward.py) and K the
roundings a term can meet, in units of 2^-24 (one fp32 rounding is half of
2^-23):
  * a chunk's Horner walk: up to 32 steps of 2 roundings;
  * the joins of chunks (4 a CTA), CTAs (up to 16 a cluster) and rounds: each a
    decay rounded (1), a product and a sum (2), powers of two being exact; in
    all 64 + 3 (20 + rounds), which 2 16 + 7 (16 + rounds) below bounds;
  * this twice over in the forward's sums (numerator and denominator of one
    quotient) and once more in (P, Q): three passes, plus 16 for the
    exponentials, reciprocals and products of the step itself (two ex2, two
    rcp at 4 each), and 2 |k| for the argument k log2(e) of e^k, whose fp32
    product and constant are off by 2^-24 relative (|k| <= 32 here beyond the
    spikes, which are the terms that dominate their own sums: +64).
What underflows: an ex2.approx flushes results below 2^-126, and so is every
fp32 product that lands there off by up to 2^-126 absolutely.  The factors it
meets on its way to a gradient of one step are a gradient |g| <= 6 and
|v| + |y| <= 12 (standard normal draws), in at most three terms:
3 72 2^-126 < 2^-118; a sum over n steps n times that (`terms`).
gw, gu, gmix: the magnitudes' sum again, plus the additions a term goes
through (32 steps, a round each, 4 warps, then the rows a group of 8 adds).
"""

import numpy as np

from tests import parity

EPS = {"f32": 2.0 ** -23, "f16": 2.0 ** -10, "bf16": 2.0 ** -7}
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -24, "bf16": 2.0 ** -133}


def k_backward(rounds: int = 1) -> float:
    return 3 * (2 * 16 + 7 * (8 + 8 + rounds)) + 16 + 64


def check(got, ref, mag, dtype: str, K: float, what: str, terms: int = 1):
    got = parity.to_f64(got)
    bound = (EPS[dtype] / 2 * np.abs(ref) + TINY[dtype] / 2 + terms * 2.0 ** -118
             + K * 2.0 ** -24 * mag * (1 + EPS[dtype] / 2))
    bad = ~(np.abs(got - ref) <= bound)  # NaN counts
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside tolerance; first at {i}: "
                             f"got {got[i]}, ref {ref[i]}, bound {bound[i]}; worst "
                             f"{np.nanmax(np.abs(got - ref) / np.maximum(bound, 1e-300)):.3g} of its bound")
