"""AdamW over parameters that lie side by side in one buffer, in any order, and
its refusal of one parameter given twice."""

import pytest
import torch

from tests.gpu_util import say

pytestmark = pytest.mark.gpu

sr = pytest.importorskip("scan_linear_rnn_amd")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bits", [8, 32])
def test_neighbours_in_one_buffer(dtype, bits):
    say(f"adamw neighbours {dtype} {bits}")
    g = torch.Generator()
    g.manual_seed(4200)
    sizes = [1, 300, 7, 5000, 20000, 256]
    ends = torch.tensor(sizes).cumsum(0).tolist()
    flat = torch.randn(ends[-1], generator=g).to("cuda", dtype)
    parts = [flat[e - n:e] for e, n in zip(ends, sizes)]
    order = [3, 0, 5, 1, 4, 2]
    alone = [parts[i].clone() for i in order]
    gs = [torch.randn(sizes[i], generator=g).cuda() for i in order]
    a, b = sr.AdamW([parts[i] for i in order], state_bits=bits), sr.AdamW(alone, state_bits=bits)
    for _ in range(2):
        a.step(gs)
        b.step(gs)
    for i, p in zip(order, alone):
        assert torch.equal(parts[i], p), i


def test_a_parameter_given_twice_is_refused():
    say("adamw tied")
    w, x = torch.ones(300, device="cuda"), torch.ones(300, device="cuda")
    g = torch.ones(300, device="cuda")
    opt = sr.AdamW([w, x, w])
    with pytest.raises(sr.ScanRNNError, match="share memory"):
        opt.step([g, g, g])
    with pytest.raises(sr.ScanRNNError, match="share memory"):
        sr.adamw_step([w, w[100:200]], [g, g[:100]], opt.m, opt.v, step=1)
    assert bool((w == 1).all() and (x == 1).all() and not opt.m.any()) and opt.steps == 0
    opt.step([g, g, None])                 # once with a gradient
    assert opt.tensor_steps == [1, 1, 0] and torch.equal(w, x)
