"""Prompts of one token for many sequences and channels: what is refused goes by the
launches that a call makes."""

import pytest
import torch

from tests.gpu_util import say
from tests.test_gpu_selective import GRADS

pytestmark = pytest.mark.gpu

sr = pytest.importorskip("scan_linear_rnn_amd")


def test_one_token_of_many_sequences():
    B, D, N = 16384, 8192, 32
    say("selective scan", B, 1, D, N)
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    n = lambda *s, dt=torch.bfloat16: torch.empty(s, device="cuda", dtype=dt).normal_(generator=g)  # noqa: E731
    u, delta, dy, Bm, Cm = n(B, 1, D), n(B, 1, D), n(B, 1, D), n(B, 1, 1, N), n(B, 1, 1, N)
    A = -n(D, N, dt=torch.float32).abs()
    rows = torch.tensor([0, 1, 8191, B - 2, B - 1], device="cuda")
    some = [t[rows] for t in (u, delta)] + [A] + [t[rows] for t in (Bm, Cm)]
    y = sr.selective_scan_forward(u, delta, A, Bm, Cm, delta_softplus=True)
    assert torch.equal(y[rows], sr.selective_scan_forward(*some, delta_softplus=True))
    got = dict(zip(GRADS, sr.selective_scan_backward(u, delta, A, Bm, Cm, dy, delta_softplus=True)))
    want = dict(zip(GRADS, sr.selective_scan_backward(*some, dy[rows], delta_softplus=True)))
    for name in ("du", "ddelta", "dB", "dC"):
        assert torch.equal(got[name][rows], want[name]), name
    torch.cuda.empty_cache()
