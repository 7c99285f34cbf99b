"""Symmetric 8-bit codes with a scale per row, and the product of codes.

TEST INFRASTRUCTURE ONLY (see the package docstring).

    scale = max |x| / 127,   q = rint(x / scale)        (ties to even)
    y[m, n] = (sum_k a[m, k] b[n, k]) a_scale[m] b_scale[n]

The scale and the quotient that is rounded are float32 numbers by definition
(NumPy's float32 division is the IEEE one): codes are integers, so where a
value lies on a tie the precision of the quotient decides, and it is part of
what is defined.  The sum is exact in int64; the scales multiply it in float64.

Pinned by tests/test_oracle_quant.py: hand-computed codes and ties, rows of
zeros and rows that are not finite, exact Fraction products.
"""

from __future__ import annotations

import numpy as np

WIDTH = 128   # stored rows are a multiple of this many codes


def quantize_rows(x):
    """(codes int8 [M, K padded with zeros to a multiple of WIDTH], scale float32 [M])."""
    x = np.asarray(x, dtype=np.float32)
    M, K = x.shape
    q = np.zeros((M, -(-K // WIDTH) * WIDTH), dtype=np.int8)
    scale = np.zeros(M, dtype=np.float32)
    for m in range(M):
        if K == 0:
            continue
        if not np.isfinite(x[m]).all():
            scale[m] = np.nan
            continue
        scale[m] = np.abs(x[m]).max() / np.float32(127)
        if scale[m] > 0:
            q[m, :K] = np.clip(np.rint(x[m] / scale[m]), -127, 127).astype(np.int8)
    return q, scale


def product(a, a_scale, b, b_scale):
    """y [M, N] in float64 from codes a [M, K], b [N, K] and their scales."""
    s = np.asarray(a, dtype=np.int64) @ np.asarray(b, dtype=np.int64).T
    return s.astype(np.float64) * (np.asarray(a_scale, np.float64)[:, None]
                                   * np.asarray(b_scale, np.float64)[None, :])
