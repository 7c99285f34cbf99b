"""A decay over many tokens is the exponential of their summed steps, whose sum must not
drift with their number.

Every channel has the same numbers: u = 0, so h_t = exp(A sum dt) h0, and dC_t is the sum of
the 64 channels' states.  Tolerance: the sum of the steps carries 16 roundings of a tile
and 4 of the tiles' sum, A log2 e two more and the exponent one, the exponential two: X (23 u) +
2 u for a decay of X; 15 tokens in a tile add 4 roundings and X / T (4 u) each, the sum
over 64 lanes 6, the start's and the products' 8: below (23 X + 80) u; each of at most 64
chunks in front adds an exponential and a product, 3 u."""

import numpy as np
import pytest
import torch

from tests.gpu_util import say

pytestmark = pytest.mark.gpu

sr = pytest.importorskip("scan_linear_rnn_amd")


@pytest.mark.parametrize("B", [1, 256])  # cut into chunks, and not
def test_equal_steps(B):
    T, D, step = 8192, 64, np.float32(0.1)
    say("selective scan backward, equal steps", B)
    full = lambda v: torch.full((B, T, D), float(v), device="cuda")  # noqa: E731
    one = torch.ones(B, T, 1, 1, device="cuda")
    A = torch.full((D, 1), -8.0 / T / 0.1, device="cuda")
    h0 = torch.ones(B, D, 1, device="cuda")
    dC = sr.selective_scan_backward(full(0), full(step), A, one, one, full(1), h0=h0)[4]
    X = -float(A[0, 0]) * float(step) * np.arange(1, T + 1)
    want = 64 * np.exp(-X)
    got = dC[:, :, 0, 0].double().cpu().numpy()
    err = np.abs(got - want) / want / 2.0 ** -24
    print("worst", err.max(), flush=True)
    assert (err <= 23 * X + 80 + (3 * 64 if B == 1 else 0)).all()
