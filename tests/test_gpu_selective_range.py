"""Chunks whose factor leaves the fp32 range while the state does not: a small state
that grows, a large one that decays.

Tolerance: test_gpu_selective.py's, with decays up to exp(106) and their inverse: 48 X u of
a term, X = 106, and 2 T + 64 roundings."""

import numpy as np
import pytest
import torch

from tests.gpu_util import say
from tests.test_gpu_selective import GRADS, U, args, case, given, host, reference

pytestmark = pytest.mark.gpu

sr = pytest.importorskip("scan_linear_rnn_amd")


def near(got, want, size, T, name):
    tol = (2 * T + 64 + 48 * 106) * U * size + 1e-37
    bad = ~(np.abs(host(got) - want) <= tol)
    assert not bad.any(), f"{name}: {bad.sum()} of {bad.size} off"


@pytest.mark.parametrize("B", [1, 256])  # cut into chunks, and not
@pytest.mark.parametrize("grows", [True, False])
def test_a_factor_out_of_range(grows, B):
    T, D, N = 200, 8, 4
    say("selective scan, a chunk's factor out of range", grows, B)
    c = case(B, T, D, N, dtype="fp32", softplus=False, bias=False)
    c["A"] = (1.0 if grows else -1.0) * (0.9 + 0.1 * torch.rand(D, N, device="cuda", generator=torch.Generator("cuda").manual_seed(3)))
    # the first 48 tokens, the first of the five chunks that one sequence is cut into, take the state by exp(+-106)
    c["delta"][:, :48] = 106 / 48
    c["delta"][:, 48:] *= 0.1
    c["u"].zero_()
    c["dy"].zero_()
    c["h0"] *= 1e-20 if grows else 1e30
    c["dh"] *= 1e-25 if grows else 1e30
    want, size = reference(c, c["dy"], c["dh"]), reference(c, c["dy"], c["dh"], True)
    y, last = sr.selective_scan_forward(*args(c), **given(c), return_last=True)
    near(last, want[1], size[1], T, "h_last")
    near(y, want[0], size[0], T, "y")
    got = dict(zip(GRADS, sr.selective_scan_backward(*args(c), c["dy"], dh_last=c["dh"], **given(c))))
    for name in ("dh0", "dA", "ddelta", "dC", "dB", "du"):
        near(got[name], want[2][name], size[2][name], T + (B * T if name == "dA" else 0), name)
