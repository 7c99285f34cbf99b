"""Products without any depth (K = 0) are zeros, up to the largest results."""

import pytest
import torch

from tests.gpu_util import say

pytestmark = pytest.mark.gpu

sr = pytest.importorskip("scan_linear_rnn_amd")


def _product(M, N, dtype):
    a, b = (torch.empty(n, 0, dtype=torch.int8, device="cuda") for n in (M, N))
    y = torch.full((M, N), -7.0, dtype=dtype, device="cuda")
    return sr.matmul_i8(a, torch.ones(M, device="cuda"), b, torch.ones(N, device="cuda"), out=y)


@pytest.mark.parametrize("M,N", [(1, 1), (300, 200), (2000, 1900), (5000, 3001), (40000, 2055)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_zeros(M, N, dtype):
    say(f"i8 no depth {M}x{N} {dtype}")
    assert not bool(_product(M, N, dtype).any())


@pytest.mark.parametrize("B,D_h", [(3, 50), (700, 600), (9000, 1025)])
def test_a_step_without_inputs(B, D_h):
    """D_in = 0: k = p = 0, so h' = h + (g(0) - h) / 2 with g(0) = 1/2, exactly
    rounded by one multiply-add."""
    say(f"i8 step without inputs {B} {D_h}")
    W = torch.empty(2 * D_h, 0, dtype=torch.int8, device="cuda")
    h0 = torch.randn(B, D_h, device="cuda")
    h = sr.mingru_step_i8(torch.empty(B, 0, device="cuda"), W, torch.ones(2 * D_h, device="cuda"), h_prev=h0)[0]
    assert bool(((h - (0.5 * (0.5 - h0) + h0)).abs() <= 2.0 ** -22 * (1 + h0.abs())).all())


def test_more_small_tiles_than_a_launch_holds():
    M, N = 1 << 20, 1 << 16     # 2^24 tiles of 64 x 64
    if torch.cuda.mem_get_info()[1] < 200 << 30:
        pytest.skip("137 GB of results")
    torch.cuda.empty_cache()
    say("i8 no depth 2^36 results")
    y = _product(M, N, torch.bfloat16)
    assert not any(bool(part.any()) for part in y.split(1 << 16))
    del y
    torch.cuda.empty_cache()
