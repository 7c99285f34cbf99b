"""Pins of oracle.quant: hand-computed codes, ties, rows that have none, exact
products; and mistakes planted in copies, each of which a pin must refuse."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import quant


def codes_pin_ok(quantize) -> bool:
    # Scale 1 (largest 127): codes are the values rounded, ties to even; the
    # second row's scale is 2^-3.
    x = np.array([[127.0, -0.5, 1.5, 2.5, -3.49], [-15.875, 0.0625, 0.125, -0.1875, 8.0]], np.float32)
    q, s = quantize(x)
    want = np.array([[127, 0, 2, 2, -3], [-127, 0, 1, -2, 64]], np.int8)
    return (q.shape == (2, 128) and np.array_equal(q[:, :5], want) and not q[:, 5:].any()
            and np.array_equal(s, np.array([1.0, 0.125], np.float32)))


def rows_without_codes_pin_ok(quantize) -> bool:
    x = np.array([[0.0, -0.0], [1.0, np.nan], [np.inf, 1.0], [1e-45, 0.0]], np.float32)
    q, s = quantize(x)
    return (not q.any() and s[0] == 0 and np.isnan(s[1]) and np.isnan(s[2])
            and s[3] == 0)   # a scale below the smallest subnormal is zero: so are the codes


def product_pin_ok(product) -> bool:
    rng = np.random.default_rng(3)
    a = rng.integers(-127, 128, (3, 128)).astype(np.int8)
    b = rng.integers(-127, 128, (4, 128)).astype(np.int8)
    sa, sb = np.array([0.5, 0.25, 3.0], np.float32), np.array([1.0, 0.125, 7.0, 0.0], np.float32)
    got = product(a, sa, b, sb)
    for m in range(3):
        for n in range(4):
            want = sum(int(x) * int(y) for x, y in zip(a[m], b[n])) * Fraction(float(sa[m])) * Fraction(float(sb[n]))
            if Fraction(got[m, n]) != want:
                return False
    return True


def test_pins_hold():
    assert codes_pin_ok(quant.quantize_rows)
    assert rows_without_codes_pin_ok(quant.quantize_rows)
    assert product_pin_ok(quant.product)
    q, s = quant.quantize_rows(np.zeros((2, 0), np.float32))
    assert q.shape == (2, 0) and np.array_equal(s, [0, 0])


def _half_up(x):
    q, s = quant.quantize_rows(x)
    live = (s > 0) & np.isfinite(s)
    out = q.copy()
    out[live, :x.shape[1]] = np.floor(x[live] / s[live, None] + 0.5).astype(np.int8)
    return out, s


def _over_128(x):
    s = np.abs(x).max(1) / np.float32(128)
    q = np.zeros((x.shape[0], 128), np.int8)
    q[:, :x.shape[1]] = np.clip(np.rint(x / s[:, None]), -127, 127)
    return q, s


def _nan_dropped(x):
    return quant.quantize_rows(np.nan_to_num(x, nan=0.0, posinf=0.0))


@pytest.mark.parametrize("pin,planted", [
    (codes_pin_ok, _half_up),
    (codes_pin_ok, _over_128),
    (rows_without_codes_pin_ok, _nan_dropped),
    (product_pin_ok, lambda a, sa, b, sb: quant.product(a, sa, b, np.roll(sb, 1))),
    (product_pin_ok, lambda a, sa, b, sb: quant.product(np.abs(a.astype(np.int64)), sa, b, sb)),
])
def test_planted_mistakes_fail(pin, planted):
    assert not pin(planted)
