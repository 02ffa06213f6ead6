"""The polynomial that the scan's softplus takes log1p(e) / e from (csrc/scan_common.cuh, softplus2), in the kernel's
fp32 arithmetic on the host: one fused multiply-add a coefficient."""
import os
import re

import numpy as np

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rwkv_wkv_recurrence_b200", "csrc",
                   "scan_common.cuh")


U = 2.0 ** -24


def _coefficients():
    text = open(SRC).read()
    body = text[text.index("softplus2"):]
    body = body[body.index("float2 r = "): body.index("return")]
    found = [np.float32(c) for c in re.findall(r"dup2\((-?[0-9.]+)f\)", body)]
    assert len(found) == 10
    return found


def _fma(a, b, c):
    # the product of two fp32 numbers is exact in 64 bits; the sum's rounding there, 2^-53, does not count
    return (a.astype(np.float64) * b.astype(np.float64) + np.float64(c)).astype(np.float32)


def test_log1p_polynomial():
    # Horner's rule rounds after each coefficient, by at most half a step of the partial result, which e <= 1 carries
    # on undiminished at most: 1 .. 0.69 (2^-25), 0.5 and 0.33 (2^-26 each), 0.25, 0.2 and 0.15 (2^-27 each), 0.11
    # (2^-28), 0.06 (2^-29), 0.02 (2^-30): together 95 x 2^-30, of a value of 0.69 or more 2.15 x 2^-24.  The product
    # with e rounds once more (2^-24), and the polynomial itself is off by its own part, taken in 64 bits.
    coef = _coefficients()
    e = np.unique(np.concatenate([
        np.linspace(0, 1, 2_000_001)[1:], np.linspace(0.95, 1, 400_001), np.exp(-np.linspace(0, 80, 400_001))
    ]).astype(np.float32))
    r, exact = np.full_like(e, coef[0]), np.full(e.shape, np.float64(coef[0]))
    for c in coef[1:]:
        r, exact = _fma(r, e, c), exact * e + np.float64(c)
    e64 = e.astype(np.float64)
    want = np.log1p(e64)
    own = (np.abs(exact * e64 - want) / want).max()
    rel = (np.abs(_fma(r, e, 0.0).astype(np.float64) - want) / want).max()
    assert own <= 0.5 * U, own / U  # the coefficients' degree and their rounding
    assert rel <= 3.15 * U + own, rel / U
