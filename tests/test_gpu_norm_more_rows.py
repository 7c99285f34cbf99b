"""The norm of more rows than its launch has workgroups, whose loop over rows takes further
turns: forward above 8192 elements (1024 workgroups), backward at all widths (1024, 512
or 256).  A row's results do not depend on its place.

Tolerance of the weight's gradient: rows of a workgroup in turn, 16 sums of workgroups per thread
and 16 of threads, below 100 roundings, and 64 of a row's own factor (test_gpu_conv_norm.py)."""

import ctypes

import pytest
import torch

from tests.gpu_util import say

pytestmark = pytest.mark.gpu

sr = pytest.importorskip("scan_linear_rnn_amd")

U = 2.0 ** -24


def random(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.empty(shape, device="cuda").normal_(generator=g)


PLACES = lambda M: (slice(0, 3), slice(1022, 1027), slice(2047, 2050), slice(M - 3, M))  # noqa: E731


@pytest.mark.parametrize("D", [8200, 10001, 16384])
@pytest.mark.parametrize("residual", [torch.float32, torch.bfloat16])
def test_forward(D, residual):
    M = 2077
    say("norm, more rows than workgroups", M, D)
    x, r, w = random(D, M, D).bfloat16(), random(D + 1, M, D).to(residual), 1 + 0.1 * random(D + 2, D)
    y, total = sr.rms_norm_forward(x, w, r)
    q, s, total_q = sr.rms_norm_quantize(x, w, r)
    assert torch.equal(total, total_q)
    plain = sr.rms_norm_forward(x, w)
    for at in PLACES(M):
        assert all(torch.equal(a[at], b) for a, b in zip((y, total), sr.rms_norm_forward(x[at], w, r[at])))
        assert all(torch.equal(a[at], b) for a, b in zip((q, s), sr.rms_norm_quantize(x[at], w, r[at])))
        assert torch.equal(plain[at], sr.rms_norm_forward(x[at], w))
    # the sum in the residual's place
    lib, p = sr.raw_library(), lambda t: ctypes.c_void_p(t.data_ptr())
    place, again = r.clone(), torch.empty_like(x)
    st = lib.rms_norm_forward(M, D, p(x), D, 1, p(place), D, int(residual == torch.bfloat16), p(w), 0, 1e-6, p(place), p(again),
                              ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert st == 0, lib.scanrnn_last_error()
    assert torch.equal(place, total) and torch.equal(again, y)


@pytest.mark.parametrize("M,D", [(9001, 100), (9001, 777), (2700, 1500), (2077, 3000), (1100, 6001), (1100, 8192), (700, 9001), (700, 16384)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_backward(M, D, dtype):
    say("norm backward, more rows than workgroups", M, D)
    total, dy, dt, w = random(D, M, D).to(dtype), random(D + 1, M, D).bfloat16(), random(D + 3, M, D).to(dtype), 1 + 0.1 * random(D + 2, D)
    dx, dw = sr.rms_norm_backward(total, w, dy, dtotal=dt)
    for at in PLACES(M):
        at = slice(min(at.start, M - 1), min(at.stop, M))
        assert torch.equal(dx[at], sr.rms_norm_backward(total[at], w, dy[at], dtotal=dt[at])[0])
    t = total.double()
    n = t * torch.rsqrt(t.square().mean(1, keepdim=True) + 1e-6)
    want, size = (dy.double() * n).sum(0), (dy.double() * n).abs().sum(0)
    assert ((dw.double() - want).abs() <= 164 * U * size).all()
    again = sr.rms_norm_backward(total, w, dy, dtotal=dt)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
