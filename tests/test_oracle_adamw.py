"""Pins of oracle.adamw: steps worked out by hand, the closed form under a
constant gradient, the float8 e4m3 values; planted mistakes must fail."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import adamw


def hand_pin_ok(step) -> bool:
    # b1 = 1/2, b2 = 3/4, t = 2, lr = 1/8, wd = 1/2, eps = 1/4; m = 1, v = 4, g = 2, p = 8:
    # m' = 3/2, v' = 3 + 1 = 4, m_hat = 2, v_hat = 4 / (7/16) = 64/7.
    p, m, v = step([8.0], [2.0], [1.0], [4.0], 2, 0.125, 0.5, 0.75, 0.25, 0.5)
    want = 8 - 0.125 * 0.5 * 8 - 0.125 * 2 / ((64 / 7) ** 0.5 + 0.25)
    return m[0] == 1.5 and v[0] == 4.0 and abs(p[0] - want) < 1e-15 * 8


def constant_gradient_pin_ok(step) -> bool:
    # From zero states a constant gradient g has m_hat = g and v_hat = g^2 at
    # every step, so each step moves p by lr g / (|g| + eps) (no decay).
    g = np.array([3.0, -0.01, 1e-9])
    p, m, v = np.zeros(3), np.zeros(3), np.zeros(3)
    for t in range(1, 6):
        p, m, v = step(p, g, m, v, t, 0.01, 0.9, 0.999, 1e-8, 0.0)
        if not np.allclose(p, -0.01 * t * g / (np.abs(g) + 1e-8), rtol=1e-9, atol=0):
            return False
    return True


def test_pins_hold():
    assert hand_pin_ok(adamw.step) and constant_gradient_pin_ok(adamw.step)


def test_codes_are_the_e4m3_values():
    vals = adamw.e4m3_values()
    assert len(vals) == 127 and np.all(np.diff(vals) > 0)
    assert vals[0] == 0 and vals[1] == adamw.TINY and vals[-1] == adamw.TOP and vals[8] == 2.0 ** -6
    assert all(Fraction(x).denominator <= 512 for x in vals)
    import torch
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(codes, vals)
    assert [adamw.span(n) for n in (0, 1, 256, 257)] == [0, 256, 256, 512]


def _planted(**swap):
    def step(p, g, m, v, t, lr, b1, b2, eps, wd):
        p, g, m, v = (np.asarray(x, dtype=np.float64) for x in (p, g, m, v))
        m = b1 * m + (1 - b1) * g
        v = b2 * v + (1 - b2) * (g * g if "square" not in swap else g)
        c1, c2 = 1 - b1 ** (t - swap.get("late", 0)), 1 - b2 ** t
        den = np.sqrt(np.abs(v) / c2) + eps if "eps" not in swap else np.sqrt(np.abs(v) / c2 + eps)
        g_wd = wd * p if "decay" not in swap else wd * m
        return p - lr * g_wd - lr * (m / c1 if "bias" not in swap else m) / den, m, v
    return step


@pytest.mark.parametrize("pin,planted", [
    (hand_pin_ok, _planted(eps=1)), (hand_pin_ok, _planted(decay=1)),
    (constant_gradient_pin_ok, _planted(bias=1)), (constant_gradient_pin_ok, _planted(square=1)),
    (hand_pin_ok, _planted(late=1)),
])
def test_planted_mistakes_fail(pin, planted):
    assert not pin(planted)


def test_unplanted_copy_passes():
    assert hand_pin_ok(_planted()) and constant_gradient_pin_ok(_planted())
