"""One AdamW step in float64, and the 8-bit form of its states.

TEST INFRASTRUCTURE ONLY (see the package docstring).

    m = b1 m + (1 - b1) g        v = b2 v + (1 - b2) g^2
    p = p - lr wd p - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)

8-bit states: blocks of 256 elements, scale = largest magnitude / 448, a code
is the float8 e4m3 value (sign, 4 exponent bits with bias 7, 3 mantissa bits,
largest 448, smallest positive 2^-9) nearest to element / scale; v is held as
its square root, and a positive root never gets the code zero.

What that rounding costs over many steps: codes of sqrt(v) are 6 to 12% apart,
and one step of b2 near 1 changes sqrt(v) by (1 - b2) / 2 of itself as a
gradient stops, which rounds back to the code that was there.  An element
then moves with its block's scale only (the largest of the 256, which is held
exactly), or by gradients so large that one step passes half a code.

Pinned by tests/test_oracle_adamw.py: hand-computed steps in exact fractions,
the closed form of a constant gradient, the 128 codes by enumeration.
"""

from __future__ import annotations

import numpy as np

BLOCK = 256
TOP = 448.0
TINY = 2.0 ** -9


def step(p, g, m, v, t, lr, b1, b2, eps, wd):
    """(p, m, v) after step t >= 1, all float64."""
    p, g, m, v = (np.asarray(x, dtype=np.float64) for x in (p, g, m, v))
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    m_hat, v_hat = m / (1 - b1 ** t), v / (1 - b2 ** t)
    return p - lr * wd * p - lr * m_hat / (np.sqrt(v_hat) + eps), m, v


def e4m3_values():
    """The 127 non-negative finite code values, ascending."""
    vals = [2.0 ** -9 * f for f in range(8)]
    for e in range(1, 16):
        vals += [2.0 ** (e - 7) * (1 + f / 8) for f in range(8) if not (e == 15 and f == 7)]
    return np.array(vals)


def held(x, positive=False):
    """What the 8-bit states hold of x, whole blocks: codes times scales."""
    blocks = np.asarray(x, dtype=np.float64).reshape(-1, BLOCK)
    scale = np.abs(blocks).max(1, keepdims=True) / TOP
    y = np.abs(blocks) / np.where(scale > 0, scale, 1.0)
    if positive:
        y = np.where(y > 0, np.maximum(y, TINY), y)
    vals = e4m3_values()
    mid = (vals[1:] + vals[:-1]) / 2                       # exact, and ties go to the even code
    i = np.searchsorted(mid, y, side="left")
    tie = (i < len(mid)) & (y == mid[np.minimum(i, len(mid) - 1)])
    return (np.sign(blocks) * vals[i + (tie & (i % 2 == 1))] * scale).reshape(np.shape(x))


def span(n):
    """A tensor's length in the state buffers."""
    return -(-n // BLOCK) * BLOCK
