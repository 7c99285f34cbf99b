"""mingru_step_i8 with its tensors side by side in one buffer, and its refusal of
a new state on top of x_t (which with few rows would be read while written)."""

import pytest
import torch

from tests.gpu_util import say

pytestmark = pytest.mark.gpu

sr = pytest.importorskip("scan_linear_rnn_amd")


@pytest.mark.parametrize("B", [1, 4, 5, 40])
def test_neighbours_and_overlaps(B):
    say(f"i8 step neighbours B={B}")
    D = 64
    g = torch.Generator(device="cuda")
    g.manual_seed(5100)
    W = sr.quantize_columns(torch.randn(D, 2 * D, device="cuda", generator=g) / 8)
    data = torch.randn(3, B, D, device="cuda", generator=g)
    x, h0 = data[0].clone(), data[2].clone()
    ref = sr.mingru_step_i8(x, *W, h_prev=h0)[0]
    h = sr.mingru_step_i8(data[0], *W, h_prev=data[2], h_next=data[1])[0]      # each begins where one ends
    assert torch.equal(h, ref) and torch.equal(data[0], x) and torch.equal(data[2], h0)
    for h_next in (data[0], data.view(-1)[1:1 + B * D].view(B, D), data.view(-1)[2 * B * D - 1:3 * B * D - 1].view(B, D)):
        with pytest.raises(sr.ScanRNNError, match="overlap"):
            sr.mingru_step_i8(data[0], *W, h_prev=data[2], h_next=h_next)
    assert torch.equal(data[0], x) and torch.equal(data[1], ref) and torch.equal(data[2], h0)
