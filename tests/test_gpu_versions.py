"""The 8-bit and AdamW calls write tensors in place where autograd can see it:
what they write counts a version up, so that a backward pass through a graph
that saved a tensor from before the call is refused, as after PyTorch's own
in-place operations, and does not silently use the new values."""

import pytest
import torch

from tests.gpu_util import say

pytestmark = pytest.mark.gpu

sr = pytest.importorskip("scan_linear_rnn_amd")


@pytest.mark.parametrize("bits", [8, 32])
def test_a_kept_graph_notices_the_step(bits):
    say(f"versions: kept graph, {bits}-bit states")
    w = torch.nn.Parameter(torch.randn(8, 8, device="cuda"))
    x = torch.randn(4, 8, device="cuda", requires_grad=True)
    opt = sr.AdamW([w], state_bits=bits)
    loss = (x @ w).square().sum()
    loss.backward(retain_graph=True)
    opt.step()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    x.grad = w.grad = None
    (x @ w).square().sum().backward()      # a graph made after the step
    assert w.grad is not None


def test_an_adamw_step_counts_what_it_writes():
    say("versions: adamw")
    ps = [torch.zeros(300, device="cuda") for _ in range(3)]
    gs = [torch.ones(300, device="cuda"), None, torch.ones(300, device="cuda")]
    for bits in (8, 32):
        opt = sr.AdamW(ps, state_bits=bits)
        written = [t for t in (ps[0], ps[2], opt.m, opt.v, opt.m_scale, opt.v_scale) if t is not None]
        others = [ps[1], gs[0], gs[2]]
        before = [t._version for t in written], [t._version for t in others]
        opt.step(gs)
        assert all(t._version > n for t, n in zip(written, before[0]))
        assert [t._version for t in others] == before[1]
    with pytest.raises(ValueError):
        opt.step(gs[:2])
    n = ps[0]._version
    with pytest.raises(sr.ScanRNNError):
        sr.adamw_step(ps, gs, opt.m, opt.v, step=0)
    assert ps[0]._version == n             # a refused call writes nothing


def test_given_outputs_count_what_is_written():
    say("versions: given outputs")
    x = torch.randn(6, 40, device="cuda")
    W = torch.randn(40, 80, device="cuda")
    q, s = sr.quantize_rows(x)
    wq, ws = sr.quantize_columns(W)
    holder = torch.zeros(7 * 80, device="cuda")
    out = holder[80:].view(6, 80)
    h = torch.zeros(6, 40, device="cuda")
    sat = torch.zeros(1, dtype=torch.int32, device="cuda")

    def counted(call, *written):
        before = [t._version for t in written]
        call()
        assert all(t._version > n for t, n in zip(written, before))

    counted(lambda: sr.quantize_rows(x, q, s), q, s)
    counted(lambda: sr.quantize_columns(W, wq, ws), wq, ws)
    counted(lambda: sr.matmul_i8(q, s, wq, ws, out=out), out, holder)     # a view counts for its base
    counted(lambda: sr.mingru_step_i8(x, wq, ws, h_prev=h, h_next=h, decay_rate=torch.zeros(40, device="cuda"),
                                      delta_t=torch.zeros(6, device="cuda"), saturated=sat), h, sat)
    counted(lambda: sr.mingru_forward_i8(x.view(2, 3, 40), wq, ws, decay_rate=torch.zeros(40, device="cuda"),
                                         delta_t=torch.zeros(2, 3, device="cuda"), saturated=sat), sat)
    assert x._version == W._version == 0


def test_inference_tensors_stay_usable():
    """Tensors made under inference_mode have no versions: they are written,
    inside and outside of it, as before."""
    say("versions: inference tensors")
    x = torch.randn(3, 64, device="cuda")
    ref_q, ref_s = sr.quantize_rows(x)
    with torch.inference_mode():
        q, s = sr.quantize_rows(x)
        q.zero_()
        sr.quantize_rows(x, q, s)
        assert torch.equal(q, ref_q)
        q.zero_()
        p = torch.ones(10, device="cuda")
    sr.quantize_rows(x, q, s)
    assert torch.equal(q, ref_q) and torch.equal(s, ref_s)
    sr.AdamW([p], lr=0.5, weight_decay=0.0).step([torch.ones(10, device="cuda")])
    assert bool((p == 0.5).all())
