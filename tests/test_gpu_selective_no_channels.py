"""No channels: the gradients of B and C, which have elements all the same, are sums of nothing."""

import ctypes

import pytest
import torch

from tests.gpu_util import say

pytestmark = pytest.mark.gpu

sr = pytest.importorskip("scan_linear_rnn_amd")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradients_of_no_channels(dtype):
    say("selective scan backward, D = 0")
    B, T, N = 2, 21, 5
    x, A = torch.zeros(B, T, 0, dtype=dtype, device="cuda"), torch.zeros(0, N, device="cuda")
    bc = torch.randn(B, T, 1, N, device="cuda").to(dtype)
    got = sr.selective_scan_backward(x, x, A, bc, bc, x)
    assert got[3].shape == got[4].shape == (B, T, 1, N)
    dB, dC = torch.full_like(bc, 7.0), torch.full_like(bc, 7.0)
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)

    def call(dB, dC):
        st = sr.raw_library().selective_scan_backward(
            B, T, 0, N, 1, None, 0, None, 0, None, 0, p(bc), N, p(bc), N, int(dtype == torch.bfloat16), None, None, None, 0, None,
            None, None, 0, None, None, None, None, dB, dC, None, None, None, None, None, 0, stream)
        assert st == 0, sr.raw_library().scanrnn_last_error()

    call(p(dB), p(dC))
    assert not dB.any() and not dC.any()
    dC.fill_(7.0)
    call(None, p(dC))
    call(None, None)
    assert not dC.any() and not got[3].any() and not got[4].any()
