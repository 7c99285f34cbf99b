"""selective_step of as many streams and channels as one launch takes."""

import pytest
import torch

from tests.gpu_util import say

pytestmark = pytest.mark.gpu

sr = pytest.importorskip("scan_linear_rnn_amd")


def test_many_streams_of_many_channels():
    B, D, N = 4096, 16384, 16
    say("selective step", B, D, N)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    n = lambda *s, dt=torch.bfloat16: torch.empty(s, device="cuda", dtype=dt).normal_(generator=g)  # noqa: E731
    u, delta, z, Bm, Cm = n(B, D), n(B, D), n(B, D), n(B, N), n(B, N)
    A, h = -n(D, N, dt=torch.float32).abs(), n(B, D, N, dt=torch.float32)
    rows = torch.tensor([0, 1, 2047, B - 2, B - 1], device="cuda")
    want = sr.selective_step(u[rows], delta[rows], A, Bm[rows], Cm[rows], z=z[rows], delta_softplus=True, h_prev=h[rows])
    y, same = sr.selective_step(u, delta, A, Bm, Cm, z=z, delta_softplus=True, h_prev=h, h_next=h)
    assert same.data_ptr() == h.data_ptr()
    assert torch.equal(y[rows], want[0]) and torch.equal(h[rows], want[1])
