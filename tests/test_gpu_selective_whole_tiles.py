"""The selective scan's walk over whole tiles, which needs more than five of them in a
chunk: prompts and gradients of long chunks, and of sequences that are not cut, against
the fp64 form."""

import pytest
import torch

from tests.gpu_util import say
from tests.test_gpu_selective import args, case, check_backward, check_forward, given, host, near, reference

pytestmark = pytest.mark.gpu

sr = pytest.importorskip("scan_linear_rnn_amd")


def chunks(B, T, D, N, G, backward):
    """How many the calls cut the tokens into, from the sizes of their workspaces (of multiples of 64 channels per group)."""
    lib = sr.raw_library()
    floats = lambda n: -(-4 * n // 256) * 256  # noqa: E731
    if not backward:
        total = lib.selective_scan_forward_workspace_size(B, T, D, N, G)
        sizes = lambda c: floats(c * B * D * N) + floats(c * B * D) if c > 1 else 0  # noqa: E731
    else:
        total = lib.selective_scan_backward_workspace_size(B, T, D, N, G)
        padded = next(n for n in (4, 8, 16, 32, 64) if n >= N)
        tiles = -(-(D // G) // 64)
        sizes = lambda c: (floats(c * B * D * N) * (2 if c > 1 else 1) + floats(c * B * D) + floats(-(-T // 16) * B * D * (N + 1)) +  # noqa: E731
                           floats(G * tiles * B * T * 2 * padded) + floats(c * B * (N + 2) * D))
    return next(c for c in range(1, T + 1) if sizes(c) == total)


@pytest.mark.parametrize("B,T,D,N,G,dtype,gated,lengths", [
    (1, 3000, 64, 16, 1, "bf16", True, [2333]), (1, 3000, 64, 16, 1, "bf16", False, None), (1, 3000, 64, 16, 1, "fp32", True, None),
    (256, 190, 64, 16, 1, "bf16", True, "odd"), (256, 190, 64, 16, 1, "fp32", False, None), (1, 1100, 64, 64, 1, "fp32", True, None),
    (1, 1100, 128, 32, 2, "bf16", True, [1099]), (1, 2100, 128, 8, 1, "fp32", True, None), (1, 1800, 66, 5, 1, "fp32", True, [1700]),
    (256, 130, 50, 12, 1, "bf16", True, None), (1, 2100, 64, 4, 1, "bf16", False, None)])
def test_long_chunks(B, T, D, N, G, dtype, gated, lengths):
    say("selective scan, long chunks", B, T, D, N, G, dtype, gated, lengths)
    for backward in (False, True):
        assert -(-T // chunks(B, T, D, N, G, backward)) > 80
    c = case(B, T, D, N, G, dtype=dtype, gated=gated, lengths=[(37 * b) % (T + 1) for b in range(B)] if lengths == "odd" else lengths)
    if lengths is not None:
        for b, n in enumerate(c["lengths"].tolist()):
            for name in ("u", "delta", "B", "C", "dy"):
                c[name][b, n:] = float("nan")
    check_forward(c)
    check_backward(c)


@pytest.mark.parametrize("at", [0, 100, 255])
def test_a_sequence_of_a_batch_is_the_sequence_alone(at):
    """In a batch of 256 the tokens are one chunk, alone several: equal up to rounding."""
    say("selective scan, alone and in a batch")
    B, T, D, N = 256, 300, 64, 16
    c = case(B, T, D, N, dtype="fp32")
    assert chunks(B, T, D, N, 1, False) == 1 and chunks(1, T, D, N, 1, False) > 1
    whole = sr.selective_scan_forward(*args(c), **given(c), return_last=True)
    one = {n: t[at:at + 1].contiguous() if torch.is_tensor(t) and t.dim() > 2 else t for n, t in c.items()}
    alone = sr.selective_scan_forward(*args(one), **given(one), return_last=True)
    size = reference(one, magnitudes=True)
    for a, b, s, name in zip(alone, whole, size, ("y", "h_last")):
        near(a, host(b[at:at + 1]), 2 * s, T, name)  # both are off by their own roundings
    again = sr.selective_scan_forward(*args(c), **given(c), return_last=True)
    assert all(torch.equal(a, b) for a, b in zip(again, whole))
