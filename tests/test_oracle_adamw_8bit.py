"""The 8-bit second moment over many steps, by its formula: what it follows and
what it does not (as the header and the AdamW docstring state it)."""

import numpy as np
import pytest

from oracle import adamw


def _roots(gradients, b2):
    """(sqrt(v) as held in 8 bits, as held exactly) after the gradients, from zeros."""
    r = v = 0.0
    for g in gradients:
        r = adamw.held(np.sqrt(b2 * r * r + (1 - b2) * g * g), positive=True)
        v = b2 * v + (1 - b2) * g * g
    return r, np.sqrt(v)


def test_held_values_by_hand():
    x = np.zeros(256)
    x[:7] = 448, 17, 19, -17, 2.0 ** -9, 2.0 ** -10, 1.5 * 2.0 ** -9
    want = np.zeros(256)
    want[:7] = 448, 16, 20, -16, 2.0 ** -9, 0, 2.0 ** -8          # ties to the even code
    assert np.array_equal(adamw.held(x), want)
    x = np.abs(x)
    want = np.abs(want)
    want[5] = 2.0 ** -9                                             # positive: never zero
    assert np.array_equal(adamw.held(x, positive=True), want)
    assert not adamw.held(np.zeros(512)).any()


@pytest.mark.parametrize("b2", [0.999, 0.99, 0.95])
def test_sizes_that_change_together_are_followed(b2):
    """All gradients eight times as large: all roots are, exactly (a power of
    two).  The largest element of a block is held exactly at every step (its code
    is 448): 3000 steps of at most four roundings of 2^-53, 2^-39 in all."""
    rng = np.random.default_rng(6000)
    size = np.exp(rng.normal(0, 1, 512))
    size[[7, 300]] = 100.0
    factor = np.concatenate([np.ones(1500), np.full(1500, 0.5)])
    gs = [size * f * rng.uniform(0.5, 1.5) for f in factor]
    held, exact = _roots(gs, b2)
    assert np.array_equal(_roots([8 * g for g in gs], b2)[0], 8 * held)
    assert np.all(np.abs(held / exact - 1)[[7, 300]] <= 2.0 ** -39)


@pytest.mark.parametrize("b2", [0.999, 0.99, 0.95])
def test_a_change_against_the_rest_of_the_block_is_not(b2):
    """Half of a block's gradients go down to a tenth, to a half or to nothing
    while the others stay: the held root stays where it was."""
    rng = np.random.default_rng(6010)
    size = np.exp(rng.normal(0, 1, 256))
    size[255] = 20.0                                                # the block's scale, unchanged
    half = np.arange(256) < 128
    before, _ = _roots([size] * 3000, b2)
    for factor in (0.0, 0.1, 0.5):
        held, exact = _roots([size] * 3000 + [np.where(half, factor * size, size)] * 3000, b2)
        assert np.all(np.abs(held / before - 1)[half] < 0.13)       # a code at most
        assert np.all(exact[half] < 0.6 * before[half])


def test_a_small_b2_decays():
    """Where a step changes the root by more than half a code it does follow."""
    size = np.ones(256)
    held, exact = _roots([size] * 100 + [np.where(np.arange(256) < 128, 0.0, 1.0)] * 300, 0.85)
    assert np.all(held[:128] < 0.01) and np.all(held[128:] > 0.9)
