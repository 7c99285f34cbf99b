"""The selective scan's softplus and its gate over the whole range of their arguments.

Softplus, u = 2^-24: with e = exp(-|x|), the exponent |x| log2 e carries two roundings (of the
constant and of the product), 2 |x| u of e, and the exponential two more; 1 + e one, given back by the correction;
the logarithm two of itself, its product with ln 2 two and the two sums two: below (2 |x| + 8) u of
the result for any x (for x > 0 the part max(x, 0) is exact).  The gate z / (1 + e^-z): 2 |z| u of e^-z,
two of the exponential, one of the sum, two of the reciprocal and two of the products: below
(2 |z| + 8) u.  Where e^-|x| is below the smallest normal number, 2^-126, it may be zero: |z| 2^-126
with |z| below 89, so 1.1e-36."""

import numpy as np
import pytest
import torch

from oracle.layers import sigmoid, softplus
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

sr = pytest.importorskip("scan_linear_rnn_amd")

U = 2.0 ** -24


def arguments():
    x = np.concatenate([np.linspace(-120, 120, 6001), np.linspace(-2, 2, 1001), [0.0, -0.0, 1e-30, -1e-30, 3e38, -3e38],
                        -np.logspace(-6, 2, 300), np.logspace(-6, 2, 300)])
    return np.resize(x, -(-len(x) // 64) * 64).astype(np.float32).astype(np.float64)


def check(got, want, x, name):
    tol = (2 * np.abs(x) + 8) * U * np.abs(want) + 1.1e-36
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= tol).all(), f"{name}: worst {np.max(err / tol):.2f} of the tolerance at {x[np.argmax(err / tol)]}"


@pytest.mark.parametrize("call", ["prompt", "token"])
def test_softplus_and_gate(call):
    say("selective scan, activations", call)
    x = arguments()
    D = len(x)
    with np.errstate(over="ignore"):
        step, silu = softplus(x), x * sigmoid(x)
    put = lambda a: torch.from_numpy(a.astype(np.float32)).to("cuda")  # noqa: E731
    one, A = torch.ones(1, 1, D, device="cuda"), torch.zeros(D, 1, device="cuda")
    bc, xs, skip = torch.ones(1, 1, 1, 1, device="cuda"), put(x).view(1, 1, D), torch.ones(D, device="cuda")
    if call == "prompt":
        _, h = sr.selective_scan_forward(one, xs, A, bc, bc, delta_softplus=True, return_last=True)
        y = sr.selective_scan_forward(one, xs, A, 0 * bc, bc, skip=skip, z=xs)
    else:
        _, h = sr.selective_step(one[:, 0], xs[:, 0], A, bc[:, 0], bc[:, 0], delta_softplus=True)
        y, _ = sr.selective_step(one[:, 0], xs[:, 0], A, 0 * bc[:, 0], bc[:, 0], skip=skip, z=xs[:, 0])
    check(h.view(-1), step, x, "softplus")   # h = exp(0) 0 + dt
    check(y.view(-1), silu, x, "gate")       # y = u silu(z)


def test_their_slopes():
    """ddelta of one token is (sum G B) u softplus'(delta), and dz is s silu'(z)."""
    say("selective scan, slopes")
    x = arguments()
    x = x[np.abs(x) <= 120]
    x = np.resize(x, -(-len(x) // 64) * 64)
    D = len(x)
    put = lambda a: torch.from_numpy(a.astype(np.float32)).to("cuda")  # noqa: E731
    one, A = torch.ones(1, 1, D, device="cuda"), torch.zeros(D, 1, device="cuda")
    bc, xs, skip = torch.ones(1, 1, 1, 1, device="cuda"), put(x).view(1, 1, D), torch.ones(D, device="cuda")
    ddelta = sr.selective_scan_backward(one, xs, A, bc, bc, one, delta_softplus=True)[1]
    check(ddelta.view(-1), sigmoid(x), x, "softplus'")
    dz = sr.selective_scan_backward(one, xs, A, 0 * bc, bc, one, skip=skip, z=xs)[6]
    p = sigmoid(x)
    # s + s z (1 - s) has terms that cancel at z = -1.278: an error goes by their sizes
    err, size = np.abs(dz.view(-1).double().cpu().numpy() - (p + x * p * (1 - p))), p + np.abs(x) * p
    assert (err <= (2 * np.abs(x) + 12) * U * size + 1.1e-36).all()
