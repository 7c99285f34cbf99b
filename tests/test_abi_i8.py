"""Refusals and sizes of the 8-bit and AdamW calls: every check runs before
anything is launched, so these need no GPU."""

import ctypes

import pytest
import torch

sr = pytest.importorskip("scan_linear_rnn_amd")
lib = sr.raw_library()

A, B, C, D = (ctypes.c_void_p(0x10000 * (i + 1)) for i in range(4))   # never dereferenced
ODD = ctypes.c_void_p(0x10008)
BAD, UNSUP, SMALL = sr.SR_ERR_INVALID_ARGUMENT, sr.SR_ERR_UNSUPPORTED, sr.SR_ERR_WORKSPACE_TOO_SMALL


def test_sizes():
    assert [lib.quantized_row_bytes(k) for k in (-1, 0, 1, 128, 129)] == [0, 0, 128, 128, 256]
    assert lib.quantized_row_bytes(2 ** 63 - 1) == 0
    assert [lib.adamw_state_elements(n) for n in (-1, 0, 1, 256, 257)] == [0, 0, 256, 256, 512]
    step = lib.mingru_step_i8_workspace_size
    assert step(256, 2048, 2048, 2048) == 256 * 2048 + 1024
    assert step(3, 100, 300, 5) == 1280 + 256 and step(0, 1, 1, 1) == 0 and step(-1, 1, 1, 1) == 0
    assert step(1 << 39, 1 << 39, 1, 1) == 0
    fwd = lib.mingru_forward_i8_workspace_size
    n32, n16 = (fwd(2, 64, 128, 128, 128, t, 0) for t in (sr.SR_F32, sr.SR_BF16))
    assert n32 - n16 == 2 * 64 * 256 * 2 and n32 % 256 == 0
    assert fwd(2, 64, 128, 128, 128, sr.SR_F32, 1) - n32 == 2 * 64 * 128 * 4
    assert fwd(2, 64, 128, 128, 128, 9, 0) == 0 and fwd(2, -1, 1, 1, 1, 0, 0) == 0


@pytest.mark.parametrize("fn", ["quantize_rows", "quantize_columns"])
@pytest.mark.parametrize("args", [
    (-1, 4, A, 4, 0, B, C), (4, -1, A, 4, 0, B, C), (4, 4, A, 3, 0, B, C), (4, 4, A, 4, 2, B, C),
    (4, 4, None, 4, 0, B, C), (4, 4, A, 4, 0, None, C), (4, 4, A, 4, 0, B, None),
    (4, 4, ctypes.c_void_p(0x10002), 4, 0, B, C), (4, 4, A, 4, 0, ODD, C), (4, 4, A, 4, 0, B, ctypes.c_void_p(0x10002)),
    (1 << 40, 1 << 40, A, 1 << 40, 0, B, C)])
def test_quantize_refusals(fn, args):
    assert getattr(lib, fn)(*args, None) == BAD
    assert lib.scanrnn_last_error()


def _mm(M=4, N=4, K=128, a=A, lda=128, sa=B, b=C, ldb=128, sb=D, y=A, ldy=4, t=0):
    return lib.matmul_i8(M, N, K, a, lda, sa, b, ldb, sb, y, ldy, t, None)


@pytest.mark.parametrize("kw", [
    dict(M=-1), dict(N=-1), dict(K=-128), dict(K=100), dict(lda=64), dict(ldb=64), dict(ldy=3), dict(t=5),
    dict(lda=136), dict(ldb=136), dict(a=None), dict(b=None), dict(sa=None), dict(sb=None), dict(y=None),
    dict(a=ODD), dict(b=ODD), dict(y=ctypes.c_void_p(0x10002)), dict(sa=ctypes.c_void_p(0x10001)),
    dict(M=1 << 60, lda=1 << 10)])
def test_product_refusals(kw):
    assert _mm(**kw) == BAD
    assert lib.scanrnn_last_error()


def test_product_depth_and_grid_limits():
    assert _mm(K=131200, lda=131200, ldb=131200) == UNSUP
    assert b"at most 131072 deep" in lib.scanrnn_last_error()
    assert _mm(M=1 << 31, N=1 << 20, ldy=1 << 20) == UNSUP


def _step(**kw):
    a = dict(B=2, D_in=4, D_h=4, D_out=4, x=A, t=0, wi=B, si=C, wo=None, so=None, rate=None, gap=None,
             log1p=0, sat=None, hp=None, hn=D, y=None, ws=A, n=1 << 20)
    a.update(kw)
    return lib.mingru_step_i8(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), BAD), (dict(D_in=1 << 50), BAD), (dict(x=None), BAD), (dict(t=7), BAD), (dict(wi=None), BAD),
    (dict(si=None), BAD), (dict(wo=B), BAD), (dict(so=C), BAD), (dict(wi=ODD), BAD), (dict(D_out=5), BAD),
    (dict(y=A), BAD), (dict(hn=None), BAD), (dict(wo=B, so=C), BAD), (dict(gap=A), BAD), (dict(sat=A), BAD),
    (dict(rate=A), BAD), (dict(rate=A, gap=B, log1p=3), BAD), (dict(ws=None), BAD), (dict(ws=ODD), BAD),
    (dict(n=16), SMALL), (dict(D_in=140000, n=1 << 30), UNSUP), (dict(D_h=140000, D_out=140000, n=1 << 30), UNSUP)])
def test_step_refusals(kw, code):
    assert _step(**kw) == code
    assert lib.scanrnn_last_error()


def _fwd(**kw):
    a = dict(B=2, T=3, D_in=4, D_h=4, D_out=4, x=A, t=1, wi=B, si=C, wo=None, so=None, rate=None, gap=None,
             log1p=0, sat=None, h0=None, y=D, last=None, ws=A, n=1 << 20)
    a.update(kw)
    return lib.mingru_forward_i8(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), BAD), (dict(B=1 << 30, T=1 << 30), BAD), (dict(x=None), BAD), (dict(t=2), BAD), (dict(wi=None), BAD),
    (dict(so=C), BAD), (dict(D_out=5), BAD), (dict(y=None), BAD), (dict(rate=A), BAD), (dict(gap=A), BAD),
    (dict(ws=None), BAD), (dict(n=16), SMALL), (dict(y=ctypes.c_void_p(0x10002)), BAD),
    (dict(D_in=140000, n=1 << 30), UNSUP)])
def test_forward_refusals(kw, code):
    assert _fwd(**kw) == code
    assert lib.scanrnn_last_error()


def _adamw(tensors=((0x10000, 0x20000, 4, 0, 0),), m=A, v=B, ms=None, vs=None, bits=32, n=1024, step=1,
           lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, wd=0.0, gs=None):
    flat = [x for p, g, k, pt, gt in tensors for x in (p, g, k, (pt & 0xFFFFFFFF) | gt << 32)]
    table = (ctypes.c_int64 * len(flat))(*flat) if flat else None
    return lib.adamw_step(len(tensors), table, m, v, ms, vs, bits, n, step, lr, b1, b2, eps, wd, gs, None)


@pytest.mark.parametrize("kw", [
    dict(bits=16), dict(step=0), dict(b1=1.0), dict(b2=-0.1), dict(lr=-1.0), dict(eps=-1.0), dict(wd=-1.0),
    dict(lr=float("nan")), dict(m=None), dict(v=None), dict(m=ODD), dict(n=100), dict(ms=C, vs=D),
    dict(bits=8), dict(bits=8, ms=C), dict(bits=8, ms=C, vs=ctypes.c_void_p(0x10001)),
    dict(gs=ctypes.c_void_p(0x10001)), dict(tensors=((0, 0x20000, 4, 0, 0),)), dict(tensors=((0x10000, 0x20000, -4, 0, 0),)),
    dict(tensors=((0x10000, 0x20000, 4, 3, 0),)), dict(tensors=((0x10000, 0x20000, 4, 0, 3),)),
    dict(tensors=((0x10002, 0x20000, 4, 0, 0),)), dict(tensors=((0x10001, 0x20000, 4, 1, 0),)),
    dict(tensors=((0x10000, 0x20000, 1 << 61, 0, 0),))])
def test_adamw_refusals(kw):
    assert _adamw(**kw) == BAD
    assert lib.scanrnn_last_error()


def test_adamw_calls_without_work_launch_nothing():
    assert _adamw(tensors=()) == sr.SR_OK
    assert _adamw(tensors=((0, 0, 0, 0, 0),), m=None, v=None, n=0) == sr.SR_OK
    assert _adamw(tensors=((0x10000, 0, 4, 0, 0),)) == sr.SR_OK        # no gradient


def test_adamw_grid_limit_is_checked_before_any_launch():
    big = 1 << 40   # more workgroups than one launch holds
    tensors = tuple((0x10000, 0x20000, 4, 0, 0) for _ in range(100)) + ((0x10000, 0x20000, big, 0, 0),)
    assert _adamw(tensors=tensors, n=big * 2) == UNSUP


def test_python_binding_refuses():
    x = torch.zeros(4, 128)
    q = torch.zeros(4, 128, dtype=torch.int8)
    for call in (lambda: sr.quantize_rows(x), lambda: sr.quantize_columns(x), lambda: sr.matmul_i8(q, x, q, x),
                 lambda: sr.mingru_step_i8(x, q, x), lambda: sr.mingru_forward_i8(x.view(1, 4, 128), q, x),
                 lambda: sr.adamw_step([x], [x], x, x, step=1), lambda: sr.adamw_step([x], [], x, x, step=1)):
        with pytest.raises((ValueError, TypeError)):
            call()
    with pytest.raises((ValueError, TypeError)):
        sr.quantize_rows(q)
    with pytest.raises(ValueError):
        sr.AdamW([x], state_bits=16)
