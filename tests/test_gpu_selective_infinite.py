"""An infinite input of the selective scan: its channel's results are the infinities
that the formula gives, for any number of states, also where they do not fill the
lanes and waves that hold them; and no other channel's gradients feel it."""

import pytest
import torch

from tests.gpu_util import say
from tests.test_gpu_selective import GRADS, args, case, given

pytestmark = pytest.mark.gpu

sr = pytest.importorskip("scan_linear_rnn_amd")

INF = float("inf")


@pytest.mark.parametrize("D", [70, 72])   # rows that are and are not taken whole
@pytest.mark.parametrize("N", [1, 3, 4, 5, 8, 9, 12, 16, 17, 20, 32, 33, 40, 64])
def test_an_infinite_input(N, D):
    say("selective scan, infinite u", N, D)
    for gated in (True, False):
        c = case(2, 120, D, N, dtype="fp32", gated=gated)
        for name in ("B", "C", "skip", "z", "h0"):  # every term of one sign
            if c[name] is not None:
                c[name].abs_()
        clean = sr.selective_scan_forward(*args(c), **given(c), return_last=True)
        c["u"][1, 5, 3] = INF
        y, last = sr.selective_scan_forward(*args(c), **given(c), return_last=True)
        assert (y[1, 5:, 3] == INF).all() and (last[1, 3] == INF).all()
        y[1, 5:, 3] = clean[0][1, 5:, 3]
        last[1, 3] = clean[1][1, 3]
        assert torch.equal(y, clean[0]) and torch.equal(last, clean[1])


@pytest.mark.parametrize("N", [1, 3, 9, 16, 20, 40, 64])
def test_gradients_of_other_channels(N):
    say("selective scan, gradients around an infinite u", N)
    c = case(2, 40, 70, N, dtype="fp32")
    clean = dict(zip(GRADS, sr.selective_scan_backward(*args(c), c["dy"], dh_last=c["dh"], **given(c))))
    c["u"][1, 5, 3] = INF
    got = dict(zip(GRADS, sr.selective_scan_backward(*args(c), c["dy"], dh_last=c["dh"], **given(c))))
    assert not torch.isfinite(got["dC"][1, 5:]).any() and not torch.isfinite(got["dB"][1, 5]).any()
    got["dC"][1, 5:], got["dB"][1, 5] = clean["dC"][1, 5:], clean["dB"][1, 5]
    for name in ("ddelta", "dz"):
        assert not torch.isfinite(got[name][1, 5:, 3]).any(), name
        got[name][1, 5:, 3] = clean[name][1, 5:, 3]
    for name in ("dA", "dskip", "dbias"):
        assert not torch.isfinite(got[name][3]).any(), name
        got[name][3] = clean[name][3]
    for name in GRADS:
        assert torch.equal(got[name], clean[name]), name
