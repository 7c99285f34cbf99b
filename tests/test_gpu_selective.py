"""The selective scan, its gradients and its single-token step against the fp64
form (oracle/layers.py).

Tolerance, with u = 2^-24: every result is a sum of products of factors that
each carry a few roundings, so an error goes by the same computation on the sizes of all
terms (nothing cancels there).  A term passes at most 2 T roundings on its way through
the states (forwards and back) and 64 in steps, gates and sums; its decays
carry the error of their exponents: a step dt = softplus(x) is off by (2.5 |x| + 8) u
(the sum and the exponential's argument are rounded) and A log2 e by 3 u more, so
exp(-X) is off by X (2.5 |x| + 11 + L) u, where L roundings come from a chunk's
summed steps (at most 16, of partial sums that grow: half of them on average).  With
|x| <= 8 that is below 48 X u; X is at most 87 before the term leaves the fp32 range, and in
these cases at most XMAX.  bf16 results are rounded once more: 2^-8 of the value."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import layers
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

sr = pytest.importorskip("scan_linear_rnn_amd")

U, XMAX, TINY = 2.0 ** -24, 40.0, 1e-30
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
GRADS = ("du", "ddelta", "dA", "dB", "dC", "dskip", "dz", "dbias", "dh0")


def host(t):
    return None if t is None else t.detach().double().cpu().numpy()


def case(B, T, D, N, G=1, dtype="bf16", gated=True, skip=True, bias=True, h0=True, lengths=None, softplus=True, seed=0):
    rng = np.random.default_rng([77, B, T, D, N, G, seed])
    dt = DTYPES[dtype]

    def put(a, t=torch.float32):
        return torch.from_numpy(np.asarray(a, dtype=np.float32)).to("cuda").to(t)

    c = dict(u=put(rng.standard_normal((B, T, D)), dt), B=put(rng.standard_normal((B, T, G, N)), dt),
             C=put(rng.standard_normal((B, T, G, N)), dt))
    # steps of about 0.01 to 0.1; without the softplus they are given as they are
    if softplus:
        c["delta"] = put(rng.uniform(-4.5, -2.2, (B, T, D)) - (rng.uniform(-1, 1, 1) if bias else 0), dt)
    else:
        c["delta"] = put(rng.uniform(0.005, 0.1, (B, T, D)), dt)
    c["A"] = put(-rng.uniform(0.05, 1.2, (D, N)))
    c["skip"] = put(rng.standard_normal(D)) if skip else None
    c["z"] = put(rng.standard_normal((B, T, D)), dt) if gated else None
    c["bias"] = put(rng.uniform(-0.3, 0.3, D) if softplus else rng.uniform(0, 0.01, D)) if bias else None
    c["h0"] = put(rng.standard_normal((B, D, N))) if h0 else None
    c["lengths"] = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    c["dy"], c["dh"] = put(rng.standard_normal((B, T, D)), dt), put(rng.standard_normal((B, D, N)))
    c["softplus"] = softplus
    return c


def given(c):
    return dict(skip=c["skip"], z=c["z"], delta_bias=c["bias"], delta_softplus=c["softplus"], h0=c["h0"], lengths=c["lengths"])


def args(c):
    return c["u"], c["delta"], c["A"], c["B"], c["C"]


def reference(c, dy=None, dh=None, magnitudes=False):
    return layers.selective(*(host(t) for t in args(c)), skip=host(c["skip"]), z=host(c["z"]), bias=host(c["bias"]),
                            softplus_on=c["softplus"], h0=host(c["h0"]),
                            lengths=None if c["lengths"] is None else c["lengths"].cpu().numpy(), dy=host(dy), dh_last=host(dh),
                            magnitudes=magnitudes)


def near(got, want, size, T, name):
    tol = (2 * T + 64 + 48 * XMAX) * U * size + TINY
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(want)
    g = host(got)
    assert g.shape == want.shape, name
    bad = ~(np.abs(g - want) <= tol)
    assert not bad.any(), f"{name}: {bad.sum()} of {bad.size}, worst {np.max(np.abs(g - want) / tol):.2f} of the tolerance"


def check_forward(c):
    y, last = sr.selective_scan_forward(*args(c), **given(c), return_last=True)
    want, size = reference(c), reference(c, magnitudes=True)
    T = c["u"].shape[1]
    near(y, want[0], size[0], T, "y")
    near(last, want[1], size[1], T, "h_last")
    return y, last


def check_backward(c, dh=True):
    dh = c["dh"] if dh else None
    got = dict(zip(GRADS, sr.selective_scan_backward(*args(c), c["dy"], dh_last=dh, **given(c))))
    want, size = reference(c, c["dy"], dh)[2], reference(c, c["dy"], dh, True)[2]
    absent = {"dskip": "skip", "dz": "z", "dbias": "bias", "dh0": "h0"}
    rows = c["u"].shape[0] * c["u"].shape[1]
    for name in GRADS:
        if name in absent and c[absent[name]] is None:
            assert got[name] is None, name
            continue
        # sums over tokens add their own chain: 16 slots, chunks and sequences
        near(got[name], want[name], size[name], c["u"].shape[1] + (rows if name in ("dA", "dskip", "dbias") else 0), name)
    return got


SHAPES = [  # B, T, D, N, G
    (2, 37, 24, 16, 1), (1, 1, 5, 1, 1), (3, 16, 64, 4, 1), (2, 17, 65, 3, 1), (1, 15, 130, 8, 2), (2, 33, 66, 7, 3),
    (1, 50, 20, 17, 1), (2, 20, 6, 32, 2), (1, 40, 9, 33, 1), (2, 19, 70, 64, 1), (1, 160, 7, 16, 1), (1, 331, 192, 16, 1),
    (4, 64, 1, 2, 1)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_scan_and_gradients(shape, dtype):
    say("selective scan", shape, dtype)
    c = case(*shape, dtype=dtype)
    check_forward(c)
    check_backward(c)


@pytest.mark.parametrize("off", ["gated", "skip", "bias", "h0", "softplus", "all"])
def test_absent_operands(off):
    say("selective scan without", off)
    names = ["gated", "skip", "bias", "h0", "softplus"] if off == "all" else [off]
    c = case(2, 150, 40, 16, dtype="fp32", **{n: False for n in names})
    check_forward(c)
    check_backward(c, dh=off != "all")


@pytest.mark.parametrize("T,lengths", [(37, [37, 0, 1, 20, 16]), (200, [0, 200, 130, 64, 17]), (20, [-3, 25, 20, 1, 0])])
def test_ragged_batches_ignore_what_stands_behind(T, lengths):
    say("selective scan, lengths", lengths)
    c = case(5, T, 70, 16, dtype="fp32", lengths=lengths)
    for b, n in enumerate(lengths):
        n = min(max(n, 0), T)
        for name in ("u", "delta", "B", "C", "z", "dy"):
            c[name][b, n:] = float("nan")
    y, _ = check_forward(c)
    got = check_backward(c)
    for b, n in enumerate(lengths):
        n = min(max(n, 0), T)
        assert not y[b, n:].any()
        for name in ("du", "ddelta", "dB", "dC", "dz"):
            assert not got[name][b, n:].any(), name


def test_no_tokens_pass_the_state():
    say("selective scan, T = 0")
    c = case(2, 0, 6, 4, dtype="fp32")
    y, last = sr.selective_scan_forward(*args(c), **given(c), return_last=True)
    assert y.shape == (2, 0, 6) and torch.equal(last, c["h0"])
    got = dict(zip(GRADS, sr.selective_scan_backward(*args(c), c["dy"], dh_last=c["dh"], **given(c))))
    assert torch.equal(got["dh0"], c["dh"])
    assert not any(got[n].any() for n in ("dA", "dskip", "dbias"))
    c = case(0, 5, 6, 4, dtype="fp32")
    y, last = sr.selective_scan_forward(*args(c), **given(c), return_last=True)
    assert y.shape == (0, 5, 6) and last.shape == (0, 6, 4)
    got = dict(zip(GRADS, sr.selective_scan_backward(*args(c), c["dy"], **given(c))))
    assert got["dA"].shape == (6, 4) and not got["dA"].any() and not got["dbias"].any()


def test_rows_of_wider_buffers_and_odd_addresses():
    """u and z as halves of one projection, delta, B and C as parts of another, at odd elements."""
    say("selective scan, strided rows")
    for B, T in ((2, 45), (1, 45), (3, 1)):
        D, N = 37, 5
        c = case(B, T, D, N, dtype="bf16")
        xz = torch.cat([c["u"], c["z"]], 2)
        pad = torch.zeros(B, T, 1, dtype=torch.bfloat16, device="cuda")
        dbc = torch.cat([pad, c["delta"], c["B"][:, :, 0], c["C"][:, :, 0], pad, pad], 2)
        want = sr.selective_scan_forward(*args(c), **given(c), return_last=True)
        grads = sr.selective_scan_backward(*args(c), c["dy"], dh_last=c["dh"], **given(c))
        v = dict(c, u=xz[..., :D], z=xz[..., D:], delta=dbc[..., 1:1 + D], B=dbc[..., 1 + D:1 + D + N],
                 C=dbc[..., 1 + D + N:1 + D + 2 * N])
        got = sr.selective_scan_forward(*args(v), **given(v), return_last=True)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        dy = c["dy"].transpose(0, 1).contiguous().transpose(0, 1)
        again = sr.selective_scan_backward(*args(v), dy, dh_last=c["dh"], **given(v))
        for name, a, b in zip(GRADS, again, grads):
            assert torch.equal(a.flatten(), b.flatten()), name
        assert again[3].shape == v["B"].shape


def test_a_prompt_in_parts_is_the_whole():
    """The state carries over: two calls, and a token at a time, against one call."""
    say("selective scan in parts")
    c = case(2, 90, 48, 16, dtype="fp32")
    kw = given(c)
    y, last = sr.selective_scan_forward(*args(c), **kw, return_last=True)
    size = reference(c, magnitudes=True)
    cut = lambda a, b: [t[:, a:b] if t.dim() > 2 else t for t in args(c)]  # noqa: E731
    h = c["h0"]
    out = []
    for a, b in ((0, 31), (31, 90)):
        kw.update(z=c["z"][:, a:b], h0=h)
        part, h = sr.selective_scan_forward(*cut(a, b), **kw, return_last=True)
        out.append(part)
    near(torch.cat(out, 1), host(y), size[0], 90, "y in parts")
    h = c["h0"].clone()
    one = dict(skip=c["skip"], delta_bias=c["bias"], delta_softplus=True)
    for t in range(90):
        tok = [x[:, t] if x.dim() > 2 else x for x in args(c)]
        y_t, same = sr.selective_step(*tok, z=c["z"][:, t], h_prev=h, h_next=h, **one)
        assert same.data_ptr() == h.data_ptr()
        near(y_t, host(y[:, t]), size[0][:, t], 90, f"token {t}")
    near(h, host(last), size[1], 90, "state after tokens")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("B,D,N,G", [(1, 1, 1, 1), (3, 10, 16, 2), (2, 33, 3, 1), (5, 7, 64, 1), (2, 12, 36, 3), (1, 9, 33, 1),
                                     (300, 20, 8, 1), (2, 6, 4, 1)])
def test_single_tokens(B, D, N, G, dtype):
    say("selective step", B, D, N, G, dtype)
    c = case(B, 1, D, N, G, dtype=dtype)
    kw = dict(skip=c["skip"], z=c["z"][:, 0], delta_bias=c["bias"], delta_softplus=True)
    tok = [t[:, 0] if t.dim() > 2 else t for t in args(c)]
    y, h = sr.selective_step(*tok, h_prev=c["h0"], **kw)
    want, size = reference(c), reference(c, magnitudes=True)
    near(y, want[0][:, 0], size[0][:, 0], 1, "y")
    near(h, want[1], size[1], 1, "h")
    y0, h0 = sr.selective_step(*tok, **kw)
    c["h0"] = None
    near(h0, reference(c)[1], reference(c, magnitudes=True)[1], 1, "h from zero")
    if G == 1:
        flat = [t.squeeze(1) if t.dim() == 3 else t for t in tok]
        y1, _ = sr.selective_step(*flat, **kw)
        assert torch.equal(y1, y0)


@pytest.mark.parametrize("B,D,N,G", [(67, 2048, 16, 1), (70, 512, 33, 2), (257, 1024, 8, 4), (131, 4096, 1, 1)])
def test_single_tokens_of_many_streams(B, D, N, G):
    """Several streams per thread, a number of them that leaves some threads without."""
    test_single_tokens(B, D, N, G, "bf16")


def test_strong_decay_and_large_steps():
    """Steps that wipe the state, and decays that underflow."""
    say("selective scan, strong decay")
    c = case(2, 70, 20, 16, dtype="fp32")
    c["delta"][:, ::7] = 30.0
    c["A"] = c["A"] * 20
    y, last = sr.selective_scan_forward(*args(c), **given(c), return_last=True)
    want, size = reference(c), reference(c, magnitudes=True)
    # a decay off by X (2.5 * 30 + 11 + 16) u, where e^-X X stays below 0.4: the rest as above
    near(y, want[0], size[0] * 2, 70, "y")
    near(last, want[1], size[1] * 2, 70, "h")
    assert all(torch.isfinite(t).all() for t in sr.selective_scan_backward(*args(c), c["dy"], **given(c)))


@pytest.mark.parametrize("N", [9, 12, 16])
def test_a_step_from_an_infinite_state(N):
    """Lanes without a state add nothing, whatever the others hold."""
    say("selective step, infinite state", N)
    c = case(2, 1, 5, N, dtype="fp32", gated=False)
    tok = [t[:, 0] if t.dim() > 2 else t for t in args(c)]
    c["h0"][1, 3, 0] = float("inf")
    c["C"].abs_()
    y, h = sr.selective_step(*tok, skip=c["skip"], delta_bias=c["bias"], delta_softplus=True, h_prev=c["h0"])
    want, size = reference(c), reference(c, magnitudes=True)
    assert y[1, 3] == float("inf") and h[1, 3, 0] == float("inf")
    ok = np.isfinite(want[0][:, 0])
    assert ok.sum() == 9
    assert (np.abs(host(y) - want[0][:, 0])[ok] <= (2 + 64 + 48 * XMAX) * U * size[0][:, 0][ok]).all()


def test_a_rate_of_minus_infinity():
    """Such a state forgets at once; the steps of zero behind a sequence's end leave it all the same."""
    say("selective scan, A = -inf")
    for T in (40, 200):
        c = case(3, T, 70, 16, dtype="fp32", lengths=[T, 21, 0])
        c["A"][3, 2] = c["A"][65, 15] = -1e30  # exp(-1e30 dt) is zero in 64 bits too
        want, size = reference(c, c["dy"], c["dh"]), reference(c, c["dy"], c["dh"], True)
        c["A"][3, 2] = c["A"][65, 15] = float("-inf")
        y, last = sr.selective_scan_forward(*args(c), **given(c), return_last=True)
        near(y, want[0], size[0], T, "y")
        near(last, want[1], size[1], T, "h_last")
        got = dict(zip(GRADS, sr.selective_scan_backward(*args(c), c["dy"], dh_last=c["dh"], **given(c))))
        for name in GRADS:
            near(got[name], want[2][name], size[2][name], T + (3 * T if name in ("dA", "dskip", "dbias") else 0), name)
        tok = [t[:, 0] if t.dim() > 2 else t for t in args(c)]
        y1, h1 = sr.selective_step(*tok, skip=c["skip"], z=c["z"][:, 0], delta_bias=c["bias"], delta_softplus=True, h_prev=c["h0"])
        near(y1[:2], want[0][:2, 0], size[0][:2, 0], 1, "token")
        assert torch.isfinite(h1).all()


@pytest.mark.parametrize("shape", [(1, 300, 130, 64, 2), (2, 180, 10, 6, 2), (1, 200, 37, 33, 1), (1, 150, 66, 20, 2),
                                   (230, 140, 5, 16, 1)])
def test_long_sequences_of_odd_widths(shape):
    """Cut into chunks, or too many for it, where rows are not taken whole."""
    say("selective scan", shape)
    c = case(*shape, dtype="bf16")
    check_forward(c)
    check_backward(c)


def test_outputs_at_an_odd_element():
    """y where no wide store may go, through the C entry point."""
    say("selective scan, y at an odd element")
    B, T, D, N = 2, 30, 64, 16
    c = case(B, T, D, N, dtype="bf16")
    want = sr.selective_scan_forward(*args(c), **given(c))
    buf = torch.full((B * T * D + 2,), 7.0, dtype=torch.bfloat16, device="cuda")
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    lib = sr.raw_library()
    st = lib.selective_scan_forward(B, T, D, N, 1, p(c["u"]), D, p(c["delta"]), D, p(c["z"]), D, p(c["B"]), N, p(c["C"]), N, 1,
                                    p(c["A"]), p(c["skip"]), p(c["bias"]), 1, p(c["h0"]), None, p(buf[1:]), None, None, 0,
                                    ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert st == 0, lib.scanrnn_last_error()
    assert torch.equal(buf[1:-1].view(B, T, D), want)
    assert buf[0] == 7 and buf[-1] == 7


def test_rows_past_four_gigabytes():
    """Rows as far apart as they may be (2^25 elements): offsets pass 2^32 elements, and the results 2^32 bytes."""
    say("selective scan, rows 2^25 elements apart")
    T, D, N = 140, 9, 5
    c = case(1, T, D, N, dtype="bf16")
    far = torch.empty(1, T, 1 << 25, dtype=torch.bfloat16, device="cuda")
    assert far.numel() > 1 << 32
    v, at = dict(c), (1 << 25) - 64
    for name in ("u", "delta", "z", "B", "C", "dy"):
        flat = c[name].reshape(1, T, -1)
        part = far[..., at:at + flat.shape[2]]
        part.copy_(flat)
        v[name] = part.unsqueeze(2) if name in ("B", "C") else part
        at += flat.shape[2]
    want = sr.selective_scan_forward(*args(c), **given(c), return_last=True)
    got = sr.selective_scan_forward(*args(v), **given(v), return_last=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    grads = sr.selective_scan_backward(*args(c), c["dy"], dh_last=c["dh"], **given(c))
    again = sr.selective_scan_backward(*args(v), v["dy"], dh_last=c["dh"], **given(v))
    for name, a, b in zip(GRADS, again, grads):
        assert torch.equal(a.flatten(), b.flatten()), name
    del far, v
    say("selective scan, large results")
    B, T, D, N = 45, 100, 1 << 20, 1
    u = torch.randn(B, T, D, dtype=torch.bfloat16, device="cuda")
    A, bc = -torch.rand(D, N, device="cuda"), torch.randn(B, T, 1, N, dtype=torch.bfloat16, device="cuda")
    y = sr.selective_scan_forward(u, u, A, bc, bc, delta_softplus=True)
    assert y.numel() > 1 << 32
    part = slice(B - 2, B)
    assert torch.equal(y[part], sr.selective_scan_forward(u[part], u[part], A, bc[part], bc[part], delta_softplus=True))
    dA_all = sr.selective_scan_backward(u, u, A, bc, bc, u, delta_softplus=True)
    for whole, own in zip(dA_all[:2] + dA_all[3:5], range(4)):
        some = sr.selective_scan_backward(u[part], u[part], A, bc[part], bc[part], u[part], delta_softplus=True)
        assert torch.equal(whole[part], (some[:2] + some[3:5])[own]), own
    del u, y, dA_all, whole, some
    torch.cuda.empty_cache()


def test_growing_states_from_zero():
    """A positive rate over a chunked sequence: the chunk's factor overflows, a zero state stays zero."""
    say("selective scan, growth")
    c = case(1, 400, 8, 4, dtype="fp32", h0=False)
    c["A"] = c["A"].abs() * 400
    c["u"].zero_()
    y, last = sr.selective_scan_forward(*args(c), **given(c), return_last=True)
    assert not y.any() and not last.any()


def test_a_nan_stays_in_its_channel_and_sequence():
    say("selective scan, NaN")
    c = case(3, 60, 70, 16, dtype="fp32")
    clean = sr.selective_scan_forward(*args(c), **given(c))
    c["u"][1, 30, 65] = float("nan")
    y = sr.selective_scan_forward(*args(c), **given(c))
    assert torch.isnan(y[1, 30:, 65]).all()
    y[1, 30:, 65] = clean[1, 30:, 65]
    assert torch.equal(y, clean)


def test_results_repeat_and_do_not_depend_on_the_batch():
    say("selective scan, repeated")
    c = case(3, 300, 128, 16, dtype="bf16")
    a = sr.selective_scan_backward(*args(c), c["dy"], dh_last=c["dh"], **given(c))
    b = sr.selective_scan_backward(*args(c), c["dy"], dh_last=c["dh"], **given(c))
    for name, x, y in zip(GRADS, a, b):
        assert torch.equal(x, y), name


def test_autograd_gives_the_backward_call():
    say("selective scan, autograd")
    c = case(2, 40, 24, 16, dtype="bf16")
    leaves = {n: c[n].clone().requires_grad_() for n in ("u", "delta", "A", "B", "C", "skip", "z", "bias", "h0")}
    y, last = sr.selective_scan(*(leaves[n] for n in ("u", "delta", "A", "B", "C")), skip=leaves["skip"], z=leaves["z"],
                                delta_bias=leaves["bias"], delta_softplus=True, h0=leaves["h0"], return_last=True)
    torch.autograd.backward([y, last], [c["dy"], c["dh"]])
    want = sr.selective_scan_backward(*args(c), c["dy"], dh_last=c["dh"], **given(c))
    for n, w in zip(leaves, want[:5] + (want[5], want[6], want[7], want[8])):
        assert torch.equal(leaves[n].grad, w) and leaves[n].grad.dtype == leaves[n].dtype, n
    y = sr.selective_scan(leaves["u"], c["delta"], c["A"], c["B"], c["C"])
    (g,) = torch.autograd.grad(y.sum(), leaves["u"], create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def test_captured_calls_replay():
    say("selective scan, graph")
    c = case(2, 200, 64, 16, dtype="bf16")
    tok = [t[:, 0].contiguous() if t.dim() > 2 else t for t in args(c)]
    h = c["h0"].clone()

    def work():
        y, last = sr.selective_scan_forward(*args(c), **given(c), return_last=True)
        grads = sr.selective_scan_backward(*args(c), c["dy"], dh_last=c["dh"], **given(c))
        step = sr.selective_step(*tok, skip=c["skip"], delta_bias=c["bias"], delta_softplus=True, h_prev=c["h0"], h_next=h)
        return [y, last, *grads, *step]

    eager = [t.clone() for t in work()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        on_stream = work()
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(on_stream, eager))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = work()
    for rep in range(3):
        junk = torch.randn(1 << 18, device="cuda").sum()
        torch.cuda.synchronize()
        for t in out:
            t.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, eager)), rep
        del junk


def test_two_streams_at_once():
    """Calls in flight together do not share what they work in."""
    say("selective scan, two streams")
    cases = [case(1, 700, 192, 16, dtype="bf16", seed=k) for k in range(2)]

    def work(c):
        return sr.selective_scan_backward(*args(c), c["dy"], dh_last=c["dh"], **given(c)) + (
            sr.selective_scan_forward(*args(c), **given(c)),)

    want = [[t.clone() for t in work(c)] for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    out = [[], []]
    for _ in range(4):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                out[k].append(work(cases[k]))
    torch.cuda.synchronize()
    for k in range(2):
        for got in out[k]:
            assert all(torch.equal(a, b) for a, b in zip(got, want[k])), k


def test_given_state_counts_a_version():
    c = case(2, 1, 8, 16, dtype="fp32")
    tok = [t[:, 0] if t.dim() > 2 else t for t in args(c)]
    h = torch.zeros(2, 8, 16, device="cuda")
    before = h._version
    sr.selective_step(*tok, h_prev=h, h_next=h)
    assert h._version > before


def test_refused():
    say("selective scan, refusals")
    c = case(2, 9, 12, 4, G=2, dtype="bf16")
    kw = given(c)

    def bad(exc=(ValueError, TypeError), **changed):
        v = dict(c, **changed)
        with pytest.raises(exc):
            sr.selective_scan_forward(*args(v), **given(v))

    bad(u=c["u"].half())
    bad(delta=c["delta"].float())
    bad(delta=c["delta"][:, :-1])
    bad(A=c["A"][:-1])
    bad(A=c["A"].bfloat16())
    bad(B=c["B"][..., :-1])
    bad(B=c["B"][:, :, :1])
    bad(z=c["z"][..., 1:])
    bad(skip=c["skip"].double())
    bad(h0=c["h0"][:1])
    bad(lengths=torch.tensor([1, 2], device="cuda"))
    bad(lengths=torch.tensor([1], dtype=torch.int32, device="cuda"))
    bad(u=c["u"].cpu())
    five = torch.zeros(2, 9, 5, 4, dtype=torch.bfloat16, device="cuda")
    bad(B=five, C=five)
    wide = torch.zeros(2, 9, 1, 65, dtype=torch.bfloat16, device="cuda")
    bad(sr.ScanRNNError, A=torch.zeros(12, 65, device="cuda"), B=wide, C=wide, h0=None)
    with pytest.raises(ValueError):
        sr.selective_scan_backward(*args(c), c["dy"], workspace=torch.empty(16, dtype=torch.uint8, device="cuda"), **kw)
    h = torch.zeros(2 * 12 * 4 + 4, device="cuda")
    tok = [t[:, 0] if t.dim() > 2 else t for t in args(c)]
    with pytest.raises(sr.ScanRNNError, match="same buffer"):
        sr.selective_step(*tok, h_prev=h[:96].view(2, 12, 4), h_next=h[4:].view(2, 12, 4))
