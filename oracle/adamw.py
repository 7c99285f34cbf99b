"""One AdamW step in float64, and the 8-bit form of its states.

TEST INFRASTRUCTURE ONLY (see the package docstring).

    m = b1 m + (1 - b1) g        v = b2 v + (1 - b2) g^2
    p = p - lr wd p - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)

8-bit states: blocks of 256 elements, scale = largest magnitude / 448, a code
is the float8 e4m3 value (sign, 4 exponent bits with bias 7, 3 mantissa bits,
largest 448, smallest positive 2^-9) nearest to element / scale; v is held as
its square root, and a positive root never gets the code zero.

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


def span(n):
    """A tensor's length in the state buffers."""
    return -(-n // BLOCK) * BLOCK
