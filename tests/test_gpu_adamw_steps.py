"""AdamW counts steps for each tensor: one whose first gradient comes late
starts with the bias correction of its own first step.

Tolerances as in test_gpu_adamw.py: the decay moves p by three roundings (2^-22
|p|), the update carries 2^-19 of itself with |m| in place of m."""

import numpy as np
import pytest
import torch

from oracle import adamw
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

sr = pytest.importorskip("scan_linear_rnn_amd")

HYPER = dict(lr=3e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.1)


def _np(t):
    return t.detach().double().cpu().numpy()


def _same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("bits", [8, 32])
def test_a_late_gradient_starts_at_its_own_first_step(bits):
    say(f"adamw late gradient {bits}")
    g = torch.Generator()
    g.manual_seed(4100)
    early, late = (torch.randn(700, generator=g).cuda() for _ in range(2))
    alone = late.clone()
    opt = sr.AdamW([early, late], state_bits=bits, **HYPER)
    for _ in range(60):
        opt.step([torch.randn(700, generator=g).cuda(), None])
    assert torch.equal(late, alone)
    fresh = sr.AdamW([alone], state_bits=bits, **HYPER)
    m = v = np.zeros(700)
    (b1, b2), lr = HYPER["betas"], HYPER["lr"]
    for t in range(1, 5):
        grad = torch.randn(700, generator=g).cuda()
        p0 = _np(late)
        opt.step([torch.randn(700, generator=g).cuda(), grad])
        fresh.step([grad])
        assert torch.equal(late, alone), t
        if bits == 32:
            size = b1 * np.abs(m) + (1 - b1) * np.abs(_np(grad))
            p, _, v1 = adamw.step(p0, _np(grad), m, v, t, lr, b1, b2, HYPER["eps"], HYPER["weight_decay"])
            update = lr / (1 - b1 ** t) * size / (np.sqrt(v1 / (1 - b2 ** t)) + HYPER["eps"])
            assert np.all(np.abs(_np(late) - p) <= 2.0 ** -22 * np.abs(p0) + 2.0 ** -19 * update), t
            m, v = _np(opt.m)[768:1468], _np(opt.v)[768:1468]      # the states that the kernel holds
    assert _same(opt.m[768:], fresh.m) and _same(opt.v[768:], fresh.v)


@pytest.mark.parametrize("bits", [8, 32])
def test_gradients_that_come_and_go(bits):
    """Each tensor moves as in an optimizer of its own that is stepped only
    where it has a gradient, bit for bit; more tensors than one launch holds."""
    say(f"adamw come and go {bits}")
    g = torch.Generator()
    g.manual_seed(4110)
    ps = [torch.randn(1 + 53 * i % 900, generator=g).cuda() for i in range(90)]
    one = [p.clone() for p in ps]
    opt = sr.AdamW(ps, state_bits=bits, **HYPER)
    singles = [sr.AdamW([p], state_bits=bits, **HYPER) for p in one]
    for k in range(6):
        gs = [torch.randn(p.shape, generator=g).cuda() if (k + i) % (1 + i % 4) == 0 else None
              for i, p in enumerate(ps)]
        opt.step(gs)
        for o, grad in zip(singles, gs):
            if grad is not None:
                o.step([grad])
    for i, (a, b) in enumerate(zip(ps, one)):
        assert torch.equal(a, b), i
    assert _same(opt.m, torch.cat([o.m.view(torch.uint8) for o in singles]))
    assert _same(opt.v, torch.cat([o.v.view(torch.uint8) for o in singles]))
    assert opt.tensor_steps == [o.steps for o in singles]


def test_counters():
    say("adamw counters")
    ps = [torch.ones(5, device="cuda"), torch.ones(6, device="cuda")]
    gs = [torch.ones_like(p) for p in ps]
    opt = sr.AdamW(ps)
    assert opt.steps == 0
    opt.step([None, None])
    assert opt.steps == 0 and opt.tensor_steps == [0, 0]
    opt.step(gs)
    opt.step([gs[0], None])
    assert opt.steps == 2 and opt.tensor_steps == [2, 1]
    for wrong in ([gs[0]], [gs[0], gs[0]], [gs[0].cpu(), gs[1]]):
        before = [p.clone() for p in ps]
        with pytest.raises(ValueError):
            opt.step(wrong)
        assert opt.tensor_steps == [2, 1] and all(torch.equal(a, b) for a, b in zip(ps, before))
    opt.steps = 7                         # all of them, as after loading states
    assert opt.tensor_steps == [7, 7]
    opt.step(iter(gs))
    assert opt.tensor_steps == [8, 8]
    opt.step([None, gs[1]])
    saved = opt.tensor_steps
    assert saved == [8, 9] and opt.steps == 9
    again = sr.AdamW([p.clone() for p in ps])
    again.m.copy_(opt.m), again.v.copy_(opt.v)
    again.tensor_steps = saved            # resumed: the same steps from here
    opt.step(gs), again.step(gs)
    assert all(torch.equal(a, b) for a, b in zip(ps, again.params)) and again.tensor_steps == [9, 10]
    with pytest.raises(ValueError):
        opt.tensor_steps = [1]
    m, v = torch.zeros(512, device="cuda"), torch.zeros(512, device="cuda")
    assert sr.adamw_step(ps, [None, gs[1]], m, v, step=[0, 3]) == 1 and not m[:256].any() and m[256:].any()
    for wrong in ([1], [1, 2, 3], [1, 0], 1.5, [1, 1.5]):
        with pytest.raises((ValueError, TypeError, sr.ScanRNNError)):
            sr.adamw_step(ps, gs, m, v, step=wrong)
    empty = sr.AdamW([])
    empty.step([])
    assert empty.steps == 0
