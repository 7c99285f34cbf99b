"""The quantised layer's parallel mode and its token loop with bf16
activations.  The loop keeps the products k and p in fp32, the parallel mode
rounds them to bf16 (2^-8 relative, half an ulp) before the gates: with z =
sigma(k), g = g(p) the states differ by e_t = (1 - z) e_{t-1} + z dg + (g - h)
dz, |dg| <= 2^-8 |p| (g rises by at most 1), |dz| <= 1.05 z (1 - z) 2^-8 |k|, so
never by more than 2^-8 (|p| + 1.05 |k| |g - h|) at its largest; 1e-4 of the
largest state is the scan's own fp32 tolerance."""

import pytest
import torch

from tests.gpu_util import say

pytestmark = pytest.mark.gpu

sr = pytest.importorskip("scan_linear_rnn_amd")


@pytest.mark.parametrize("dim", [16, 96, 513])
@pytest.mark.parametrize("decay", [False, True])
def test_prompt_and_tokens_carry_the_same_states(dim, decay):
    say(f"i8 bf16 modes {dim} decay={decay}")
    g = torch.Generator()
    g.manual_seed(5200)
    q = sr.MinGRU(dim, W_out=False, generator=g, decay_rate=0.05 if decay else None).quantized()
    x = torch.randn(3, 60, dim, generator=g).to("cuda", torch.bfloat16)
    gaps = torch.rand(3, 60, generator=g).cuda() if decay else None
    states = q(x, delta_t=gaps)
    h, loop = torch.zeros(3, dim, device="cuda"), []
    for t in range(60):
        h = q(x[:, t], h, delta_t=gaps[:, t] if decay else None)
        loop.append(h)
    loop = torch.stack(loop, 1)
    k, p = sr.matmul_i8(*sr.quantize_rows(x), q.W_in, q.W_in_scale).chunk(2, dim=-1)
    top = lambda v: float(v.abs().max())  # noqa: E731
    gap = top(torch.where(p >= 0, p + 0.5, torch.sigmoid(p))) + top(loop)
    bound = 2.0 ** -8 * (top(p) + 1.05 * top(k) * gap) + 1e-4 * top(loop)
    assert top(states - loop) <= bound, (top(states - loop), bound)
    first = q(x[:, :30], None, return_next_prev_hidden=True, delta_t=gaps[:, :30] if decay else None)[1]
    rest = q(x[:, 30:], first, delta_t=gaps[:, 30:] if decay else None)   # a prompt in two parts
    assert top(rest - states[:, 30:]) <= 1e-4 * (1 + top(states))
