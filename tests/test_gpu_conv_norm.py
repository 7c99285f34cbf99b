"""The short causal convolution and the root-mean-square norm against their fp64
forms (oracle/layers.py).

Tolerances, with u = 2^-24 and sizes of all terms from the oracle: a sum of K
products and the SiLU of it is off by less than 64 u of the terms' sizes (the
logistic's argument, |c| log2 e below 64, is rounded once, and |silu'| < 1.1); a gradient of
the filter adds the chain of a run (at most 64 tokens), of 16 partial sums and of the runs
that one thread adds, at most `rows` in all.  A norm's sum of squares is a chain of at
most 32 elements and 10 halvings, half of whose error reaches the result: 64 u, twice
that for its gradient, whose sum over rows adds at most `rows` more.  bf16
results are rounded once more: 2^-8 of the value; a code is off by half of its scale."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import layers
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

sr = pytest.importorskip("scan_linear_rnn_amd")

U = 2.0 ** -24
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


def host(t):
    return None if t is None else t.detach().double().cpu().numpy()


def near(got, want, size, roundings, name):
    tol = roundings * U * size + 1e-30
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(want)
    g = host(got)
    assert g.shape == want.shape, name
    bad = ~(np.abs(g - want) <= tol)
    assert not bad.any(), f"{name}: {bad.sum()} of {bad.size}, worst {np.max(np.abs(g - want) / tol):.2f} of the tolerance"


def put(a, t=torch.float32):
    return torch.from_numpy(np.asarray(a, dtype=np.float32)).to("cuda").to(t)


def conv_case(B, T, D, K, dtype="bf16", w_dtype=None, bias=True, state=True, lengths=None):
    rng = np.random.default_rng([78, B, T, D, K])
    dt, wt = DTYPES[dtype], DTYPES[w_dtype or dtype]
    c = dict(x=put(rng.standard_normal((B, T, D)), dt), w=put(rng.standard_normal((D, K)), wt),
             bias=put(rng.standard_normal(D), wt) if bias else None,
             state=put(rng.standard_normal((B, K - 1, D)), dt) if state else None,
             lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    return c, put(rng.standard_normal((B, T, D)), dt), put(rng.standard_normal((B, K - 1, D)), dt)


def conv_reference(c, silu, dy=None, dlast=None, magnitudes=False):
    return layers.conv(host(c["x"]), host(c["w"]), host(c["bias"]), silu, host(c["state"]),
                       None if c["lengths"] is None else c["lengths"].cpu().numpy(), host(dy), host(dlast), magnitudes)


def check_conv(c, dy, dlast, silu):
    kw = dict(silu=silu, state=c["state"], lengths=c["lengths"])
    y, last = sr.causal_conv_forward(c["x"], c["w"], c["bias"], return_last=True, **kw)
    want, size = conv_reference(c, silu, dy, dlast), conv_reference(c, silu, dy, dlast, True)
    near(y, want[0], size[0], 64, "y")
    assert np.array_equal(host(last), want[1])
    got = dict(zip(("dx", "dw", "dbias", "dstate"),
                   sr.causal_conv_backward(c["x"], c["w"], dy, c["bias"], dlast=dlast, **kw)))
    rows = c["x"].shape[0] * c["x"].shape[1]
    for name, have in got.items():
        if have is None:
            assert c[{"dbias": "bias", "dstate": "state"}[name]] is None
            continue
        near(have, want[2][name], size[2][name], 128 + min(rows, 64 + 16 + rows // 16), name)
    return y, got


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("B,T,D,K", [(2, 37, 24, 4), (1, 1, 1, 1), (3, 2, 7, 4), (1, 9, 8, 2), (2, 100, 33, 3), (1, 5, 130, 8),
                                     (2, 21, 5, 5), (1, 70, 12, 6), (2, 8, 16, 7), (1, 3, 4, 1), (1, 400, 1001, 4)])
def test_conv_and_gradients(B, T, D, K, dtype, silu):
    say("conv", B, T, D, K, dtype, silu)
    check_conv(*conv_case(B, T, D, K, dtype), silu)


@pytest.mark.parametrize("dtype,w_dtype,bias,state", [("bf16", "fp32", True, False), ("fp32", "bf16", False, True),
                                                      ("bf16", "bf16", False, False)])
def test_conv_types_and_absent_operands(dtype, w_dtype, bias, state):
    say("conv", dtype, w_dtype, bias, state)
    c, dy, dlast = conv_case(2, 30, 20, 4, dtype, w_dtype, bias, state)
    check_conv(c, dy, dlast, True)
    check_conv(c, dy, None, True)


@pytest.mark.parametrize("T,lengths", [(20, [20, 0, 1, 2, 11]), (3, [3, 0, 1, 2, -1]), (70, [99, 64, 65, 4, 3])])
def test_ragged_conv_ignores_what_stands_behind(T, lengths):
    say("conv, lengths", lengths)
    c, dy, dlast = conv_case(5, T, 19, 4, "fp32", lengths=lengths)
    for b, n in enumerate(lengths):
        n = min(max(n, 0), T)
        c["x"][b, n:] = float("nan")
        dy[b, n:] = float("nan")
    y, got = check_conv(c, dy, dlast, True)
    for b, n in enumerate(lengths):
        n = min(max(n, 0), T)
        assert not y[b, n:].any() and not got["dx"][b, n:].any()


def test_conv_without_tokens_passes_the_state():
    say("conv, T = 0")
    c, dy, dlast = conv_case(2, 0, 6, 4, "fp32")
    y, last = sr.causal_conv_forward(c["x"], c["w"], c["bias"], state=c["state"], return_last=True)
    assert y.shape == (2, 0, 6) and torch.equal(last, c["state"])
    dx, dw, db, dstate = sr.causal_conv_backward(c["x"], c["w"], dy, c["bias"], state=c["state"], dlast=dlast)
    assert torch.equal(dstate, dlast) and not dw.any() and not db.any()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("B,D,K", [(1, 1, 1), (3, 16, 4), (2, 9, 3), (300, 24, 4), (2, 8, 8), (1, 40, 2)])
def test_conv_tokens_are_the_prompt(B, D, K, dtype):
    """Token after token, in place, gives the prompt's outputs and state bit for bit."""
    say("conv step", B, D, K, dtype)
    c, _, _ = conv_case(B, 6, D, K, dtype)
    y, last = sr.causal_conv_forward(c["x"], c["w"], c["bias"], silu=True, state=c["state"], return_last=True)
    state = c["state"].clone()
    for t in range(6):
        y_t, same = sr.causal_conv_step(c["x"][:, t], c["w"], c["bias"], silu=True, state=state, state_next=state)
        assert torch.equal(y_t, y[:, t]) and same.data_ptr() == state.data_ptr()
    assert torch.equal(state, last)
    y0, s0 = sr.causal_conv_step(c["x"][:, 0], c["w"], c["bias"])
    want = sr.causal_conv_forward(c["x"][:, :1], c["w"], c["bias"], return_last=True)
    assert torch.equal(y0, want[0][:, 0]) and torch.equal(s0, want[1])


def test_conv_rows_of_a_wider_buffer():
    say("conv, strided rows")
    c, dy, dlast = conv_case(2, 33, 21, 4, "bf16")
    wide = torch.cat([c["x"][..., :3], c["x"], c["x"]], 2)
    for a, b in zip(sr.causal_conv_forward(wide[..., 3:24], c["w"], c["bias"], silu=True, return_last=True),
                    sr.causal_conv_forward(c["x"], c["w"], c["bias"], silu=True, return_last=True)):
        assert torch.equal(a, b)
    for a, b in zip(sr.causal_conv_backward(wide[..., 3:24], c["w"], wide[..., 24:], c["bias"])[:3],
                    sr.causal_conv_backward(c["x"], c["w"], c["x"], c["bias"])[:3]):
        assert torch.equal(a, b)


def norm_case(M, D, dtype, rdtype, w_dtype=None):
    rng = np.random.default_rng([79, M, D])
    x = put(rng.standard_normal((M, D)) * 2, DTYPES[dtype])
    r = put(rng.standard_normal((M, D)) * 3, DTYPES[rdtype]) if rdtype else None
    return x, r, put(1 + 0.1 * rng.standard_normal(D), DTYPES[w_dtype or dtype]), rng


WIDTHS = [1, 7, 8, 16, 127, 128, 129, 255, 300, 512, 1001, 1024, 2048, 2049, 5000, 8192, 16384]


@pytest.mark.parametrize("dtype,rdtype", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32"), ("fp32", "bf16"), ("bf16", ""),
                                          ("fp32", "")])
@pytest.mark.parametrize("D", WIDTHS)
def test_norm_codes_and_gradients(D, dtype, rdtype):
    M = 67 if D <= 2048 else 5
    say("norm", M, D, dtype, rdtype)
    x, r, w, rng = norm_case(M, D, dtype, rdtype, "fp32" if D % 2 else None)
    eps = 1e-5
    total = x if r is None else (x.float() + r.float()).to(r.dtype)
    out = sr.rms_norm_forward(x, w, r, eps=eps)
    y = out if r is None else out[0]
    if r is not None:
        assert torch.equal(out[1], total)
    want = layers.norm(host(total), host(w), eps)
    near(y, want, np.abs(want), 64, "y")
    q, scale, *more = sr.rms_norm_quantize(x, w, r, eps=eps)
    if r is not None:
        assert torch.equal(more[0], total)
    assert q.shape == (M, sr.quantized_row_bytes(D)) and not q[:, D:].any()
    top = np.abs(want).max(1) / 127
    assert (np.abs(host(scale) - top) <= 66 * U * top).all()
    off = np.abs(host(q)[:, :D] * host(scale)[:, None] - want)
    assert (off <= host(scale)[:, None] * (0.5 + 127 * 132 * U)).all()
    dy, dt = put(rng.standard_normal((M, D)), x.dtype), put(rng.standard_normal((M, D)), total.dtype)
    for d in (dt, None):
        dx, dw = sr.rms_norm_backward(total, w, dy, dtotal=d, eps=eps)
        _, dx_want, dw_want = layers.norm(host(total), host(w), eps, host(dy), host(d))
        _, dx_size, dw_size = layers.norm(host(total), host(w), eps, host(dy), host(d), True)
        near(dx, dx_want, dx_size, 160, "dx")
        near(dw, dw_want, dw_size, 160 + M, "dw")


def test_norm_of_zeros_infinities_and_no_rows():
    say("norm, edges")
    x = torch.zeros(3, 40, device="cuda")
    w = torch.ones(40, device="cuda")
    assert not sr.rms_norm_forward(x, w).any()
    q, s = sr.rms_norm_quantize(x, w)
    assert not q.any() and not s.any()
    x[1, 3], x[2, 4] = float("inf"), float("nan")
    q, s = sr.rms_norm_quantize(x, w)
    assert s[0] == 0 and torch.isnan(s[1:]).all() and not q.any()
    none = torch.zeros(0, 40, device="cuda")
    assert sr.rms_norm_forward(none, w).shape == (0, 40) and sr.rms_norm_quantize(none, w)[0].shape == (0, 128)
    dx, dw = sr.rms_norm_backward(none, w, none)
    assert dx.shape == (0, 40) and not dw.any()


def test_norm_shapes_and_strided_rows():
    say("norm, strides")
    x, r, w, _ = norm_case(12, 50, "bf16", "fp32")
    flat = sr.rms_norm_forward(x, w, r)
    cube = sr.rms_norm_forward(x.view(3, 4, 50), w, r.view(3, 4, 50))
    wide = torch.cat([x, x], 1)[:, 50:]
    again = sr.rms_norm_forward(wide, w, r)
    for a, b, c in zip(flat, cube, again):
        assert torch.equal(a, b.view(12, 50)) and torch.equal(a, c)
    q, s, t = sr.rms_norm_quantize(x.view(3, 4, 50), w, r.view(3, 4, 50))
    assert q.shape == (3, 4, 128) and s.shape == (3, 4) and t.shape == (3, 4, 50)


def test_the_sum_may_take_the_residuals_place():
    say("norm, total in place")
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    lib = sr.raw_library()
    for D in (9, 200, 2048, 5000, 10000):
        x, r, w, _ = norm_case(37, D, "bf16", "fp32")
        want, total = sr.rms_norm_forward(x, w, r)
        y = torch.empty_like(x)
        st = lib.rms_norm_forward(37, D, p(x), D, 1, p(r), D, 0, p(w), 1, 1e-6, p(r), p(y),
                                  ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        assert st == 0, lib.scanrnn_last_error()
        assert torch.equal(r, total) and torch.equal(y, want), D


def test_rows_past_four_gigabytes():
    """Inputs and results of more than 2^32 elements: their last rows are those of a small call."""
    say("norm and convolution, large tensors")
    rows = (1 << 32) // 2048 + 1000
    x = torch.randn(rows, 2048, dtype=torch.bfloat16, device="cuda")
    w = torch.rand(2048, device="cuda").bfloat16()
    part = slice(rows - 70, rows)
    y, total = sr.rms_norm_forward(x, w, x)
    for big, small in zip((y, total), sr.rms_norm_forward(x[part], w, x[part])):
        assert torch.equal(big[part], small)
    dx = sr.rms_norm_backward(y, w, total)[0]
    assert torch.equal(dx[part], sr.rms_norm_backward(y[part], w, total[part])[0])
    del dx, total
    q, s, _ = sr.rms_norm_quantize(x, w, x)
    for big, small in zip((q, s), sr.rms_norm_quantize(x[part], w, x[part])):
        assert torch.equal(big[part], small)
    del q, s
    f = torch.randn(2048, 4, device="cuda").bfloat16()
    x3, y3 = x.view(1, rows, 2048), y.view(1, rows, 2048)
    out = sr.causal_conv_forward(x3, f, silu=True)
    assert torch.equal(out[:, part], sr.causal_conv_forward(x3[:, part], f, silu=True, state=x3[:, rows - 73:rows - 70]))
    dx = sr.causal_conv_backward(x3, f, y3, silu=True)[0]
    some = sr.causal_conv_backward(x3[:, part], f, y3[:, part], silu=True, state=x3[:, rows - 73:rows - 70])[0]
    assert torch.equal(dx[:, part], some)
    del x, y, x3, y3, out, dx, some
    torch.cuda.empty_cache()


def test_many_rows_of_each_width_repeat():
    """More rows than the grid has workgroups; a row's result does not depend on its place."""
    say("norm, many rows")
    for D in (33, 192, 2048):
        M = 20011
        g = torch.Generator(device="cuda")
        g.manual_seed(D)
        x = torch.empty((M, D), device="cuda").normal_(generator=g).bfloat16()
        w = torch.empty(D, device="cuda").uniform_(0.5, 1.5, generator=g)
        y = sr.rms_norm_forward(x, w)
        for at in (0, 9999, M - 3):
            assert torch.equal(y[at:at + 3], sr.rms_norm_forward(x[at:at + 3], w))
        dx, dw = sr.rms_norm_backward(x, w, x)
        dx2, dw2 = sr.rms_norm_backward(x, w, x)
        assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
        xd = x.double()
        inv = torch.rsqrt(xd.square().mean(1, keepdim=True) + 1e-6)
        want, size = (xd * xd * inv).sum(0), (xd * xd * inv).abs().sum(0)
        # chains of rows per workgroup and of workgroups per thread: below 200 roundings
        assert ((dw.double() - want).abs() <= 400 * U * size).all()


def test_autograd_of_a_block():
    """norm with residual, convolution and scan as a layer has them: autograd against the fp64 forms' gradients."""
    say("block, autograd")
    rng = np.random.default_rng(80)
    B, T, D, N, K, eps = 2, 30, 16, 8, 4, 1e-5
    v = {n: rng.standard_normal(s) for n, s in dict(x=(B, T, D), r=(B, T, D), w=D, cw=(D, K), cb=D, delta=(B, T, D), Bm=(B, T, 1, N),
                                                    Cm=(B, T, 1, N), skip=D, z=(B, T, D)).items()}
    v["A"], v["delta"] = -rng.uniform(0.1, 1, (D, N)), rng.uniform(-4, -2, (B, T, D))
    t = {n: put(a).requires_grad_() for n, a in v.items()}
    v = {n: host(a) for n, a in t.items()}
    y, total = sr.rms_norm(t["x"], t["w"], t["r"], eps=eps)
    c = sr.causal_conv(y, t["cw"], t["cb"], silu=True)
    out = sr.selective_scan(c, t["delta"], t["A"], t["Bm"], t["Cm"], skip=t["skip"], z=t["z"], delta_softplus=True)
    dout, dtot = rng.standard_normal((B, T, D)), rng.standard_normal((B, T, D))
    torch.autograd.backward([out, total], [put(dout), put(dtot)])
    dout, dtot = host(put(dout)), host(put(dtot))
    tot = host(total).reshape(-1, D)
    n_y = layers.norm(tot, v["w"], eps).reshape(B, T, D)
    c_y, _ = layers.conv(n_y, v["cw"], v["cb"])
    want, _, g = layers.selective(c_y, v["delta"], v["A"], v["Bm"], v["Cm"], v["skip"], v["z"], dy=dout)
    _, _, gc = layers.conv(n_y, v["cw"], v["cb"], dy=g["du"])
    _, dx, dw = layers.norm(tot, v["w"], eps, gc["dx"].reshape(-1, D), dtot.reshape(-1, D))
    got = {n: host(a.grad) for n, a in t.items()}
    pairs = dict(x=dx.reshape(B, T, D), r=dx.reshape(B, T, D), w=dw, cw=gc["dw"], cb=gc["dbias"], delta=g["ddelta"], A=g["dA"],
                 Bm=g["dB"], Cm=g["dC"], skip=g["dskip"], z=g["dz"])
    for n, a in pairs.items():
        # three operators in fp32 of a few hundred roundings each, whose terms cancel by less than a factor of ten in norm
        assert np.linalg.norm(got[n] - a) <= 1e4 * U * np.linalg.norm(a), n
    assert np.linalg.norm(host(out) - want) <= 1e4 * U * np.linalg.norm(want)


def test_serving_in_8_bits_feeds_the_product():
    """norm to codes to the 8-bit product to convolution and scan, for a prompt and then its next token, on a second stream too."""
    say("block, 8-bit serving")
    g = torch.Generator(device="cuda")
    g.manual_seed(81)
    B, T, D, N = 2, 40, 64, 16
    n = lambda *s: torch.empty(s, device="cuda").normal_(generator=g)  # noqa: E731
    x, r, w = n(B, T + 1, D).bfloat16(), n(B, T + 1, D), 1 + 0.1 * n(D)
    W, ws = sr.quantize_columns(n(D, 2 * D) / 8)
    cw, cb, A, skip, bias = n(D, 4), n(D), -n(D, N).abs(), n(D), n(D) - 4
    dbc = n(B, T + 1, D + 2 * N).bfloat16()

    def layer(x, r, dbc, conv, scan):
        q, s, total = sr.rms_norm_quantize(x, w, r)
        xz = sr.matmul_i8(q, s, W, ws, out_dtype=torch.bfloat16)
        u, conv = conv(xz[..., :D])
        y, h = scan(u, dbc[..., :D], dbc[..., D:D + N], dbc[..., D + N:], xz[..., D:])
        return y, conv, h, total

    kw = dict(skip=skip, delta_bias=bias, delta_softplus=True)

    def prompt(m):
        return layer(x[:, :m], r[:, :m], dbc[:, :m], lambda u: sr.causal_conv_forward(u, cw, cb, silu=True, return_last=True),
                     lambda u, d, b, c, z: sr.selective_scan_forward(u, d, A, b, c, z=z, return_last=True, **kw))

    y, conv, h, total = prompt(T)
    y1, conv1, h1, _ = layer(x[:, T], r[:, T], dbc[:, T], lambda u: sr.causal_conv_step(u, cw, cb, silu=True, state=conv),
                             lambda u, d, b, c, z: sr.selective_step(u, d, A, b, c, z=z, h_prev=h, **kw))
    whole, conv2, h2, _ = prompt(T + 1)
    assert torch.equal(conv1, conv2) and torch.equal(whole[:, :T], y)
    # the same sums in another order: a few roundings of fp32, and one of bf16 that may fall the other way
    assert (h1 - h2).norm() <= 1e-5 * h2.norm() and (y1 - whole[:, T]).float().norm() <= 2.0 ** -7 * whole[:, T].float().norm()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = prompt(T + 1)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(again[0], whole) and torch.equal(again[2], h2)


def test_captured_calls_replay():
    say("conv and norm, graph")
    c, dy, dlast = conv_case(2, 300, 64, 4, "bf16")
    x, r, w, _ = norm_case(600, 192, "bf16", "fp32")
    state = c["state"].clone()

    def work():
        out = [*sr.causal_conv_forward(c["x"], c["w"], c["bias"], silu=True, state=c["state"], return_last=True)]
        out += sr.causal_conv_backward(c["x"], c["w"], dy, c["bias"], silu=True, state=c["state"], dlast=dlast)
        out += sr.causal_conv_step(c["x"][:, 0], c["w"], c["bias"], state=c["state"], state_next=state)
        out += sr.rms_norm_forward(x, w, r)
        out += sr.rms_norm_quantize(x, w, r)
        return out + list(sr.rms_norm_backward(r, w, x, dtotal=r))

    eager = [t.clone() for t in work()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        work()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = work()
    for rep in range(3):
        junk = torch.randn(1 << 18, device="cuda").sum()
        torch.cuda.synchronize()
        for t in out:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, eager)), rep
        del junk


def test_refused():
    say("conv and norm, refusals")
    c, dy, _ = conv_case(2, 9, 12, 4, "bf16")

    def bad(call, exc=(ValueError, TypeError)):
        with pytest.raises(exc):
            call()

    bad(lambda: sr.causal_conv_forward(c["x"].half(), c["w"]))
    bad(lambda: sr.causal_conv_forward(c["x"], c["w"][:-1]))
    bad(lambda: sr.causal_conv_forward(c["x"], c["w"], c["bias"].float()))
    bad(lambda: sr.causal_conv_forward(c["x"], c["w"], state=c["state"][:, 1:]))
    bad(lambda: sr.causal_conv_forward(c["x"], c["w"], lengths=torch.tensor([1, 2], device="cuda")))
    bad(lambda: sr.causal_conv_forward(c["x"], torch.zeros(12, 9, device="cuda")), sr.ScanRNNError)
    bad(lambda: sr.causal_conv_backward(c["x"], c["w"], dy.float()))
    buf = torch.zeros(2 * 3 * 12 + 12, dtype=torch.bfloat16, device="cuda")
    bad(lambda: sr.causal_conv_step(c["x"][:, 0], c["w"], state=buf[:72].view(2, 3, 12), state_next=buf[12:].view(2, 3, 12)),
        sr.ScanRNNError)
    x, r, w, _ = norm_case(4, 20, "bf16", "fp32")
    bad(lambda: sr.rms_norm_forward(x, w[:-1]))
    bad(lambda: sr.rms_norm_forward(x, w, r[:2]))
    bad(lambda: sr.rms_norm_forward(x, w.double()))
    bad(lambda: sr.rms_norm_forward(x, w, eps=-1.0), sr.ScanRNNError)
    bad(lambda: sr.rms_norm_backward(r, w, x, dtotal=x))
    wide = torch.zeros(2, 16385, device="cuda")
    bad(lambda: sr.rms_norm_forward(wide, wide[0]), sr.ScanRNNError)
