"""The AdamW step against the oracle.

Tolerances.  m and v are sums of two products with rounded constants: at most
five roundings of 2^-24 each, relative to the terms' magnitudes (taken as
2^-21).  p gets the decay (three roundings of |p|: 2^-22 |p|) and an update
whose numerator carries m's error and whose other factors a dozen roundings
(square root, division, constants): 2^-19 of the update with |m| in place of m.
A bf16 p adds 2^-8 |p|.  8-bit codes are the nearest e4m3 values: half a step,
2^-4 relative or 2^-10 of the scale below the normal range, and a positive
root below that range is raised to 2^-9 of the scale at most."""

import numpy as np
import pytest
import torch

from oracle import adamw
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

sr = pytest.importorskip("scan_linear_rnn_amd")

HYPER = dict(lr=3e-3, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1)
SIZES = [(16, 32), (1,), (255,), (256,), (257,), (1023,), (3, 1000), (64, 129), (0,), (5000,)]
TYPES = [torch.float32, torch.bfloat16]


def _np(t):
    return t.detach().double().cpu().numpy()


def _offsets(sizes):
    at, total = [], 0
    for s in sizes:
        at.append(total)
        total += adamw.span(int(np.prod(s)))
    return at, total


def _decode(code, scale):
    return _np(code).reshape(-1, 256) * _np(scale)[:, None]


def _tensors(sizes, p_type, g_type, seed):
    g = torch.Generator()
    g.manual_seed(seed)
    ps = [torch.randn(s, generator=g).to("cuda", p_type) for s in sizes]
    gs = [(torch.randn(s, generator=g) * 10.0 ** -(i % 6)).to("cuda", g_type) for i, s in enumerate(sizes)]
    return ps, gs


def _check(p0, g, p1, m0, v0, m1, v1, step, hyper, scale=1.0):
    """p1, m1, v1 against the oracle's step from p0, m0, v0 (arrays, float64)."""
    (b1, b2), lr = hyper["betas"], hyper["lr"]
    g64 = _np(g).reshape(-1) * scale
    p, m, v = adamw.step(_np(p0).reshape(-1), g64, m0, v0, step, lr, b1, b2, hyper["eps"], hyper["weight_decay"])
    size = b1 * np.abs(m0) + (1 - b1) * np.abs(g64)
    update = lr / (1 - b1 ** step) * size / (np.sqrt(v / (1 - b2 ** step)) + hyper["eps"])
    tol = 2.0 ** -22 * np.abs(_np(p0).reshape(-1)) + 2.0 ** -19 * update
    if p1.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(p)
    assert np.all(np.abs(_np(p1).reshape(-1) - p) <= tol), float(np.max(np.abs(_np(p1).reshape(-1) - p) - tol))
    if m1 is not None:
        assert np.all(np.abs(m1 - m) <= 2.0 ** -21 * size)
        assert np.all(np.abs(v1 - v) <= 2.0 ** -21 * v)
    return m, v


@pytest.mark.parametrize("p_type", TYPES)
@pytest.mark.parametrize("g_type", TYPES)
def test_fp32_states(p_type, g_type):
    say(f"adamw fp32 states {p_type} {g_type}")
    ps, gs = _tensors(SIZES, p_type, g_type, 4000)
    at, total = _offsets(SIZES)
    m, v = torch.zeros(total, device="cuda"), torch.zeros(total, device="cuda")
    for step in (1, 2, 3):
        before = [p.clone() for p in ps], _np(m), _np(v)
        sr.adamw_step(ps, gs, m, v, step=step, **HYPER)
        for i, o in enumerate(at):
            s = slice(o, o + ps[i].numel())
            _check(before[0][i], gs[i], ps[i], before[1][s], before[2][s], _np(m)[s], _np(v)[s], step, HYPER)
            assert not m[s.stop:o + adamw.span(ps[i].numel())].any()    # the spans' tails stay zero


def _check_codes(code, scale, target, positive):
    """code, scale of whole blocks against the float64 values they stand for."""
    blocks = target.reshape(-1, 256)
    s_ref = np.abs(blocks).max(1) / adamw.TOP
    assert np.all(np.abs(_np(scale) - s_ref) <= 2.0 ** -20 * s_ref)
    err = np.abs(_decode(code, scale) - blocks)
    low = (2.0 ** -9 if positive else 2.0 ** -10) * s_ref[:, None]
    assert np.all(err <= (2.0 ** -4 + 2.0 ** -18) * np.abs(blocks) + low)
    if positive:
        live = (blocks > 0) & (s_ref[:, None] > 0)
        assert np.all(_np(code).reshape(-1, 256)[live] >= adamw.TINY)


@pytest.mark.parametrize("p_type", TYPES)
@pytest.mark.parametrize("g_type", TYPES)
def test_8bit_states(p_type, g_type):
    say(f"adamw 8-bit states {p_type} {g_type}")
    ps, gs = _tensors(SIZES, p_type, g_type, 4010)
    at, total = _offsets(SIZES)
    m, v = (torch.zeros(total, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
    ms, vs = torch.zeros(total // 256, device="cuda"), torch.zeros(total // 256, device="cuda")
    for step in (1, 2, 3):
        p0, m0, r0 = [p.clone() for p in ps], _decode(m, ms).reshape(-1), _decode(v, vs).reshape(-1)
        sr.adamw_step(ps, gs, m, v, m_scale=ms, v_scale=vs, step=step, **HYPER)
        for i, o in enumerate(at):
            n, end = ps[i].numel(), o + adamw.span(ps[i].numel())
            if n == 0:
                continue
            mi, vi = _check(p0[i], gs[i], ps[i], m0[o:o + n], r0[o:o + n] ** 2, None, None, step, HYPER)
            pad = np.zeros(end - o - n)
            b = slice(o // 256, end // 256)
            _check_codes(m[o:end], ms[b], np.concatenate([mi, pad]), False)
            _check_codes(v[o:end], vs[b], np.concatenate([np.sqrt(vi), pad]), True)


def test_8bit_states_are_the_formula_operation_by_operation():
    """Codes on ties are decided by float32 roundings: NumPy's float32, one
    operation at a time, gives the same codes and scales bit for bit, two
    steps on (the second step starts from the first one's codes)."""
    say("adamw 8-bit codes")
    f = np.float32
    n, (b1, b2) = 40 * 256, HYPER["betas"]
    g = torch.Generator()
    g.manual_seed(4015)
    p = torch.randn(n, generator=g).cuda()
    opt = sr.AdamW([p], state_bits=8, **HYPER)
    vals = adamw.e4m3_values().astype(f)
    mid = (vals[1:].astype(np.float64) + vals[:-1]) / 2          # ties go to the even code

    def nearest(y):
        i = np.searchsorted(mid, np.abs(y).astype(np.float64), side="left")
        tie = (i < len(mid)) & (np.abs(y).astype(np.float64) == mid[np.minimum(i, len(mid) - 1)])
        i = np.where(tie & (i % 2 == 1), i + 1, i)
        return np.where(y < 0, -vals[i], vals[i]).astype(f)

    def encode(x, positive):
        x = x.reshape(-1, 256)
        s = np.abs(x).max(1) * (f(1) / f(448))
        y = x / s[:, None]
        y = np.where(x > 0, np.maximum(y, f(adamw.TINY)), y) if positive else y
        return nearest(np.minimum(np.maximum(y, f(-448)), f(448))), s

    m = v = np.zeros((40, 256), f)
    for step in (1, 2):
        grad = torch.randn(n, generator=g) * 0.01
        opt.step([grad.cuda()])
        gn = grad.numpy().reshape(-1, 256)
        m = m * f(b1) + gn * f(1 - b1)
        v = v * f(b2) + gn * gn * f(1 - b2)
        assert m.dtype == v.dtype == f
        (mc, ms), (vc, vs) = encode(m, False), encode(np.sqrt(v), True)
        for name, want, got in (("m", mc, opt.m), ("v", vc, opt.v), ("ms", ms, opt.m_scale), ("vs", vs, opt.v_scale)):
            assert np.array_equal(got.float().cpu().numpy().reshape(want.shape), want), (step, name)
        m, v = mc * ms[:, None], (vc * vs[:, None]) ** 2


@pytest.mark.parametrize("bits", [8, 32])
def test_many_tensors_and_skipped_gradients(bits):
    """More tensors than one launch's table holds, some without a gradient:
    the result is that of one call per tensor, bit for bit."""
    say(f"adamw many tensors {bits}")
    sizes = [(1 + 37 * i % 700,) for i in range(300)]
    ps, gs = _tensors(sizes, torch.float32, torch.float32, 4020)
    gs = [None if i % 7 == 3 else g for i, g in enumerate(gs)]
    one = [p.clone() for p in ps]
    opt = sr.AdamW(ps, state_bits=bits, **HYPER)
    singles = [sr.AdamW([p], state_bits=bits, **HYPER) for p in one]
    for _ in range(2):
        opt.step(gs)
        for o, g in zip(singles, gs):
            o.step([g])
    for i, (a, b) in enumerate(zip(ps, one)):
        assert torch.equal(a, b), i
    same = lambda x, y: torch.equal(x.view(torch.uint8), y.view(torch.uint8))  # noqa: E731
    assert same(opt.m, torch.cat([o.m.view(torch.uint8) for o in singles]).view(opt.m.dtype))
    assert same(opt.v, torch.cat([o.v.view(torch.uint8) for o in singles]).view(opt.v.dtype))


def test_unaligned_tensors():
    """Parameters and gradients at odd element offsets of larger buffers, and
    the elements around them untouched."""
    say("adamw unaligned")
    for p_type in TYPES:
        for n in (1, 300, 2049):
            buf = torch.full((n + 7,), 5.0, device="cuda", dtype=p_type)
            gbuf = torch.full((n + 9,), 0.25, device="cuda", dtype=p_type)
            p, g = buf[3:3 + n], gbuf[1:1 + n]
            ref = p.clone()
            for bits in (8, 32):
                a, b = sr.AdamW([p], state_bits=bits), sr.AdamW([ref], state_bits=bits)
                a.step([g])
                b.step([g.clone()])
            assert torch.equal(p, ref)
            assert bool((buf[:3] == 5).all() and (buf[3 + n:] == 5).all() and (gbuf == 0.25).all())


def test_grad_scale_and_parameters_grad():
    say("adamw grad_scale")
    ps, gs = _tensors([(300,), (8, 64)], torch.float32, torch.float32, 4030)
    at, total = _offsets([(300,), (8, 64)])
    m, v = torch.zeros(total, device="cuda"), torch.zeros(total, device="cuda")
    p0 = [p.clone() for p in ps]
    half = torch.tensor([0.5], device="cuda")
    sr.adamw_step(ps, gs, m, v, step=1, grad_scale=half, **HYPER)
    for i, o in enumerate(at):
        s = slice(o, o + ps[i].numel())
        _check(p0[i], gs[i], ps[i], np.zeros(ps[i].numel()), np.zeros(ps[i].numel()), _np(m)[s], _np(v)[s], 1,
               HYPER, scale=0.5)
    w = torch.nn.Parameter(p0[0].clone())
    (w * gs[0]).sum().backward()
    opt = sr.AdamW([w], **HYPER)
    opt.step(grad_scale=half)
    assert torch.equal(w.detach(), ps[0])
    opt.zero_grad()
    assert w.grad is None
    opt.step()                      # no gradient: nothing moves
    assert torch.equal(w.detach(), ps[0])


def test_values_that_are_not_finite():
    """fp32 states: only the element itself is lost.  8-bit states: its block."""
    say("adamw non-finite")
    for bad in (float("nan"), float("inf"), -float("inf")):
        g = torch.ones(1000, device="cuda")
        g[300] = bad
        p = torch.zeros(1000, device="cuda")
        sr.AdamW([p]).step([g])
        assert not bool(torch.isfinite(p[300])) and int(torch.isfinite(p).sum()) == 999
        q = torch.zeros(1000, device="cuda")
        opt = sr.AdamW([q], state_bits=8)
        opt.step([g])
        assert torch.equal(p, q) or torch.equal(p.isnan(), q.isnan())
        assert [bool(x) for x in opt.m_scale.isnan()] == [False, True, False, False]
        assert [bool(x) for x in opt.v_scale.isnan()] == [False, True, False, False]
        opt.step([torch.ones_like(g)])
        assert bool(q[256:512].isnan().all()) and bool(torch.isfinite(q[:256]).all() and torch.isfinite(q[512:]).all())


def test_tiny_and_vanishing_states():
    """Gradients that stop: the states decay through the subnormals without a
    NaN, and the weights stop moving apart from the weight decay."""
    say("adamw vanishing states")
    for bits in (8, 32):
        p = torch.ones(700, device="cuda")
        opt = sr.AdamW([p], lr=1e-3, weight_decay=0.0, state_bits=bits, betas=(0.3, 0.3))
        opt.step([torch.full_like(p, 1e-18)])
        zero = torch.zeros_like(p)
        for _ in range(250):
            opt.step([zero])
        assert bool(torch.isfinite(p).all()) and bool((p.sub(1).abs() < 0.02).all())
        scales = opt.m_scale if bits == 8 else opt.m
        assert bool(torch.isfinite(scales).all())
    tiny = torch.zeros(256, device="cuda")
    opt = sr.AdamW([tiny], state_bits=8)
    g = torch.full((256,), 1e-38, device="cuda")
    g[7] = 3e-40
    opt.step([g])
    assert bool(torch.isfinite(tiny).all()) and bool(torch.isfinite(opt.m.float()).all())


def test_past_2_31_elements():
    say("adamw past 2^31 elements")
    n = (1 << 31) + 1500
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    g[-1000:] = -2.0
    opt = sr.AdamW([p], lr=0.5, weight_decay=0.0, state_bits=8)
    opt.step([g])
    assert bool((p[:1000] == -0.5).all()) and bool((p[-1000:] == 0.5).all()) and bool((p[-1500:-1000] == -0.5).all())
    assert float(opt.m[n - 1].float() * opt.m_scale[(n - 1) // 256]) == pytest.approx(-0.2, rel=1e-6)


def test_8bit_training_follows_fp32_training():
    """A least-squares fit: both reach the same loss within a few percent."""
    say("adamw fit")
    g = torch.Generator()
    g.manual_seed(4040)
    A = torch.randn(256, 64, generator=g).cuda()
    target = A @ torch.randn(64, 32, generator=g).cuda()
    losses = {}
    for bits in (32, 8):
        w = torch.zeros(64, 32, device="cuda")
        opt = sr.AdamW([w], lr=0.05, weight_decay=0.0, state_bits=bits)
        for _ in range(400):
            r = A @ w - target
            opt.step([A.t() @ r / 256])
        losses[bits] = float((A @ w - target).square().mean() / target.square().mean())
    assert losses[32] < 1e-3 and losses[8] < 1e-3, losses


def test_graph_replays_match_eager():
    say("adamw graph")
    for bits in (8, 32):
        ps, gs = _tensors([(300,), (40, 70), (5,)], torch.float32, torch.float32, 4050)
        ref = [p.clone() for p in ps]
        a, b = sr.AdamW(ps, state_bits=bits), sr.AdamW(ref, state_bits=bits)
        a.step(gs), b.step(gs)             # warm-up; both at step 1
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):      # records step 2 (its number is a constant of the recording)
            a.step(gs)
        for rep in range(3):
            b.steps = 1
            b.step(gs)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(ps, ref)), rep
