"""The fp64 forms of the selective scan, the convolution and the norm: their
gradients against central differences, their recurrences against closed forms."""

import numpy as np
import pytest

from oracle import layers


def _differences(f, x, dout, h=1e-5):
    """Gradient of sum(f(x) dout) by central differences."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        old = x[i]
        x[i] = old + h
        up = f()
        x[i] = old - h
        g[i] = ((up - f()) / (2 * h) * 1.0)
        x[i] = old
    return g


def _scan_case(gated, on, ragged):
    rng = np.random.default_rng([31, gated, on, ragged])
    nb, T, D, G, N = 2, 5, 4, 2, 3
    v = dict(u=rng.standard_normal((nb, T, D)), delta=rng.uniform(0.1, 1, (nb, T, D)), A=-rng.uniform(0.2, 2, (D, N)),
             B=rng.standard_normal((nb, T, G, N)), C=rng.standard_normal((nb, T, G, N)), skip=rng.standard_normal(D),
             z=rng.standard_normal((nb, T, D)) if gated else None, bias=rng.uniform(0, 1, D), softplus_on=on,
             h0=rng.standard_normal((nb, D, N)), lengths=np.array([T, 2]) if ragged else None)
    return v, rng.standard_normal((nb, T, D)), rng.standard_normal((nb, D, N))


@pytest.mark.parametrize("gated,on,ragged", [(1, 1, 0), (0, 1, 1), (1, 0, 1)])
def test_selective_gradients_are_those_of_differences(gated, on, ragged):
    v, dy, dh = _scan_case(gated, on, ragged)
    _, _, grads = layers.selective(**v, dy=dy, dh_last=dh)

    def loss():
        y, h = layers.selective(**v)
        return float((y * dy).sum() + (h * dh).sum())

    names = {"du": "u", "ddelta": "delta", "dA": "A", "dB": "B", "dC": "C", "dskip": "skip", "dbias": "bias", "dh0": "h0"}
    if gated:
        names["dz"] = "z"
    for g, name in names.items():
        # the third derivatives are of order one: h^2 = 1e-10, and the differences' rounding 1e-16 / h
        assert np.allclose(grads[g], _differences(loss, v[name], None), rtol=1e-7, atol=1e-8), g


def test_selective_scan_of_constant_inputs_is_a_geometric_sum():
    a, T = -0.3, 40
    one = np.ones((1, T, 1))
    y, h = layers.selective(one, one * 0.5, np.full((1, 1), a), one[..., None], one[..., None], softplus_on=False)
    r = np.exp(0.5 * a)
    want = 0.5 * (1 - r ** np.arange(1, T + 1)) / (1 - r)
    assert np.allclose(y[0, :, 0], want, rtol=1e-13) and np.isclose(h[0, 0, 0], want[-1], rtol=1e-13)


@pytest.mark.parametrize("K,T,ragged", [(4, 6, 1), (3, 1, 0), (1, 4, 0), (4, 2, 0)])
def test_conv_gradients_are_those_of_differences(K, T, ragged):
    rng = np.random.default_rng([32, K, T])
    nb, D = 3, 2
    v = dict(x=rng.standard_normal((nb, T, D)), w=rng.standard_normal((D, K)), bias=rng.standard_normal(D),
             state=rng.standard_normal((nb, K - 1, D)), lengths=np.array([T, 1, 0]) if ragged else None)
    dy, dl = rng.standard_normal((nb, T, D)), rng.standard_normal((nb, K - 1, D))
    _, _, grads = layers.conv(**v, dy=dy, dlast=dl)

    def loss():
        y, last = layers.conv(**v)
        return float((y * dy).sum() + (last * dl).sum())

    for g, name in {"dx": "x", "dw": "w", "dbias": "bias", "dstate": "state"}.items():
        assert np.allclose(grads[g], _differences(loss, v[name], None), rtol=1e-7, atol=1e-8), g


def test_conv_continues_where_its_state_ends():
    rng = np.random.default_rng(33)
    x, w, b = rng.standard_normal((2, 9, 3)), rng.standard_normal((3, 4)), rng.standard_normal(3)
    whole, end = layers.conv(x, w, b)
    first, state = layers.conv(x[:, :2], w, b)
    second, last = layers.conv(x[:, 2:], w, b, state=state)
    assert np.allclose(np.concatenate([first, second], 1), whole, rtol=1e-14) and np.array_equal(last, end)


def test_norm_gradients_are_those_of_differences():
    rng = np.random.default_rng(34)
    t, w, dy, dt = rng.standard_normal((3, 5)), rng.standard_normal(5), rng.standard_normal((3, 5)), rng.standard_normal((3, 5))
    _, dx, dw = layers.norm(t, w, 1e-2, dy, dt)

    def loss():
        return float((layers.norm(t, w, 1e-2) * dy).sum() + (t * dt).sum())

    assert np.allclose(dx, _differences(loss, t, None), rtol=1e-7, atol=1e-8)
    assert np.allclose(dw, _differences(loss, w, None), rtol=1e-7, atol=1e-8)
