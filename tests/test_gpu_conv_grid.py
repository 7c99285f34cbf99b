"""The short convolution of one token for many sequences: what is refused goes by the
launches that a call makes."""

import pytest
import torch

from tests.gpu_util import say

pytestmark = pytest.mark.gpu

sr = pytest.importorskip("scan_linear_rnn_amd")


def random(*shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(len(shape))
    return torch.empty(shape, device="cuda", dtype=torch.bfloat16).normal_(generator=g)


def test_one_token_of_many_sequences():
    B, D, K = 1 << 19, 2048, 4
    say("convolution", B, 1, D, K)
    x, w = random(B, 1, D), random(D, K)
    rows = torch.tensor([0, 1, 70000, B - 2, B - 1], device="cuda")
    y = sr.causal_conv_forward(x, w, silu=True)
    assert torch.equal(y[rows], sr.causal_conv_forward(x[rows], w, silu=True))
    dx = sr.causal_conv_backward(x, w, y, silu=True)[0]
    assert torch.equal(dx[rows], sr.causal_conv_backward(x[rows], w, y[rows], silu=True)[0])
    del x, y, dx
    torch.cuda.empty_cache()


def test_a_step_of_more_than_2_32_elements():
    B, D, K = (1 << 21) + 3, 2048, 2
    say("convolution step", B, D, K)
    x, w = random(B, D), random(D, K)
    state = x.flip(0).view(B, 1, D)
    rows = torch.tensor([0, 1, 70000, B - 2, B - 1], device="cuda")
    want = sr.causal_conv_step(x[rows], w, silu=True, state=state[rows])
    y, same = sr.causal_conv_step(x, w, silu=True, state=state, state_next=state)
    assert same.data_ptr() == state.data_ptr()
    assert torch.equal(y[rows], want[0]) and torch.equal(state[rows], want[1])
    del x, state, y, same
    torch.cuda.empty_cache()
