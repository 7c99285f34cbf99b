"""An infinite input of the short convolution reaches the gradients of the taps that
it passes under, and no other."""

import numpy as np
import pytest
import torch

from tests.gpu_util import say
from tests.test_gpu_conv_norm import conv_case, conv_reference, host, near

pytestmark = pytest.mark.gpu

sr = pytest.importorskip("scan_linear_rnn_amd")


@pytest.mark.parametrize("T,lengths", [(10, None), (64, None), (30, [21]), (131, None)])
@pytest.mark.parametrize("back", [1, 2])
def test_gradient_of_the_taps(back, T, lengths):
    say("convolution backward, infinite input", T, lengths, back)
    D, K = 12, 4
    c, dy, _ = conv_case(1, T, D, K, dtype="fp32", lengths=lengths)
    end = (lengths or [T])[0]
    c["x"][0, end - back, 5] = float("inf")  # the last input is under the last tap alone, the one before under two
    dx, dw, dbias, _ = sr.causal_conv_backward(c["x"], c["w"], dy, c["bias"], state=c["state"], lengths=c["lengths"])
    # without the activation only those taps' gradients hold it: all others are those of a finite one in its place
    finite = dict(c, x=c["x"].masked_fill(torch.isinf(c["x"]), 1.0))
    want, size = conv_reference(finite, False, dy)[2], conv_reference(finite, False, dy, magnitudes=True)[2]
    hit = np.zeros((D, K), bool)
    hit[5, K - back:] = True
    assert np.isinf(host(dw)[hit]).all()
    near(torch.where(torch.from_numpy(hit).to("cuda"), 0.0, dw), np.where(hit, 0.0, want["dw"]), size["dw"], 64 + T, "dw")
    near(dx, want["dx"], size["dx"], 64, "dx")
    near(dbias, want["dbias"], size["dbias"], 64 + T, "dbias")
