"""Refusals and sizes of the selective scan's, the convolution's and the norm's
calls: every check runs before anything is launched, so these need no GPU."""

import ctypes

import pytest
import torch

sr = pytest.importorskip("scan_linear_rnn_amd")
lib = sr.raw_library()

BAD, UNSUP, SMALL, OK = sr.SR_ERR_INVALID_ARGUMENT, sr.SR_ERR_UNSUPPORTED, sr.SR_ERR_WORKSPACE_TOO_SMALL, sr.SR_OK


def at(i, off=0):
    return ctypes.c_void_p(0x10000000 * (i + 1) + off)     # never dereferenced


def test_sizes():
    f, b = lib.selective_scan_forward_workspace_size, lib.selective_scan_backward_workspace_size
    assert f(256, 512, 2048, 16, 1) == 0          # enough sequences and channels: no chunks
    assert f(1, 4096, 512, 16, 1) > 0 and f(1, 4096, 512, 16, 1) % 256 == 0
    assert b(2, 64, 128, 16, 1) > b(2, 64, 128, 8, 1) > 0
    for call in (f, b):
        for args in ((-1, 1, 1, 1, 1), (1, -1, 1, 1, 1), (1, 1, 1, 0, 1), (1, 1, 1, 65, 1), (1, 1, 6, 4, 4), (1, 1, 6, 4, 0),
                     (1 << 30, 1 << 30, 1 << 10, 4, 1)):
            assert call(*args) == 0, args
    c = lib.causal_conv_backward_workspace_size
    assert c(1, 0, 8, 4, 0) == 256 and c(2, 4, 64, 4, 1) == 2 * 5 * 64 * 4
    assert c(1, 1, 8, 9, 0) == c(1, 1, 8, 0, 0) == c(-1, 1, 8, 4, 0) == c(1, -1, 8, 4, 0) == c(1, 1, 8, 4, 3) == 0
    n = lib.rms_norm_backward_workspace_size
    assert n(1, 64) == 256 and n(0, 64) == 0 and n(-1, 64) == n(4, 0) == n(4, 16385) == 0


def scan(**kw):
    a = dict(B=2, T=64, D=8, N=4, G=2, u=at(0), ld_u=8, delta=at(1), ld_d=8, z=at(2), ld_z=8, Bm=at(3), ld_b=8, Cm=at(4), ld_c=8,
             t=0, A=at(5), skip=at(6), bias=at(7), on=1, h0=None, lengths=None, y=at(8), last=None, ws=at(9), n=1 << 20)
    a.update(kw)
    return lib.selective_scan_forward(*a.values(), None)


SHARED = [(dict(B=-1), BAD), (dict(D=-2), BAD), (dict(N=0), BAD), (dict(N=65, ld_b=200, ld_c=200), UNSUP), (dict(G=3), BAD),
          (dict(G=0), BAD), (dict(u=None), BAD), (dict(delta=None), BAD), (dict(Bm=None), BAD), (dict(Cm=None), BAD),
          (dict(A=None), BAD), (dict(ld_u=7), BAD), (dict(ld_d=7), BAD), (dict(ld_z=7), BAD), (dict(ld_b=7), BAD), (dict(ld_c=7), BAD),
          (dict(ld_u=1 << 62), BAD), (dict(t=2), BAD), (dict(on=2), BAD), (dict(u=at(0, 2)), BAD), (dict(A=at(5, 2)), BAD),
          (dict(skip=at(6, 1)), BAD), (dict(y=None), BAD), (dict(y=at(8, 2)), BAD), (dict(y=at(0)), BAD), (dict(y=at(5)), BAD),
          (dict(B=1 << 41), BAD)]


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(T=-1), BAD), (dict(lengths=at(10, 2)), BAD), (dict(h0=at(10), last=at(10)), BAD), (dict(last=at(8)), BAD),
    (dict(y=at(3, 16)), BAD), (dict(B=1, T=4096, ws=None), BAD), (dict(B=1, T=4096, ws=at(9, 8)), BAD),
    (dict(B=1, T=4096, n=64), SMALL), (dict(B=1 << 30, T=1), UNSUP), (dict(ld_u=1 << 26), UNSUP), (dict(ld_c=1 << 26), UNSUP)])
def test_scan_refusals(kw, code):
    assert scan(**kw) == code
    assert lib.scanrnn_last_error()


def test_calls_without_work_launch_nothing():
    assert scan(B=0) == OK and scan(D=0, G=1, y=None) == OK
    assert step(B=0) == OK and conv(B=0) == OK and conv(D=0) == OK and conv_step(B=0) == OK
    assert norm(M=0) == OK and codes(M=0) == OK


def step(**kw):
    a = dict(B=2, D=8, N=4, G=2, u=at(0), ld_u=8, delta=at(1), ld_d=8, z=at(2), ld_z=8, Bm=at(3), ld_b=8, Cm=at(4), ld_c=8, t=0,
             A=at(5), skip=at(6), bias=at(7), on=1, prev=at(9), next=at(9), y=at(8))
    a.update(kw)
    return lib.selective_step(*a.values(), None)


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(next=None), BAD), (dict(next=at(9, 4)), BAD), (dict(next=at(0)), BAD), (dict(y=at(9)), BAD), (dict(prev=at(9, 2)), BAD)])
def test_step_refusals(kw, code):
    assert step(**kw) == code
    assert lib.scanrnn_last_error()


def scan_backward(**kw):
    a = dict(B=2, T=64, D=8, N=4, G=2, u=at(0), ld_u=8, delta=at(1), ld_d=8, z=at(2), ld_z=8, Bm=at(3), ld_b=8, Cm=at(4), ld_c=8,
             t=0, A=at(5), skip=at(6), bias=at(7), on=1, h0=None, lengths=None, dy=at(8), ld_dy=8, dh=None, du=at(10), dd=at(11),
             dz=at(12), dB=at(13), dC=at(14), dA=at(15), dskip=at(16), dbias=at(17), dh0=None, ws=at(18), n=1 << 30)
    a.update(kw)
    return lib.selective_scan_backward(*a.values(), None)


@pytest.mark.parametrize("kw,code", [x for x in SHARED if "y" not in x[0]] + [
    (dict(T=-1), BAD), (dict(dy=None), BAD), (dict(du=None), BAD), (dict(dd=None), BAD), (dict(dB=None), BAD), (dict(dC=None), BAD),
    (dict(dA=None), BAD), (dict(dz=None), BAD), (dict(z=None), BAD), (dict(ld_dy=7), BAD), (dict(ld_dy=1 << 62), BAD),
    (dict(dy=at(8, 2)), BAD), (dict(dA=at(15, 2)), BAD), (dict(du=at(0)), BAD), (dict(du=at(11)), BAD), (dict(dskip=at(17)), BAD),
    (dict(dh=at(20), dh0=at(20)), BAD), (dict(dB=at(8)), BAD), (dict(ws=None), BAD), (dict(n=64), SMALL), (dict(ld_dy=1 << 26), UNSUP)])
def test_scan_backward_refusals(kw, code):
    assert scan_backward(**kw) == code
    assert lib.scanrnn_last_error()


def conv(**kw):
    a = dict(B=2, T=5, D=8, K=4, x=at(0), ld=8, t=0, w=at(1), bias=at(2), wt=1, silu=1, state=at(3), lengths=None, y=at(4), last=at(5))
    a.update(kw)
    return lib.causal_conv_forward(*a.values(), None)


def conv_backward(**kw):
    a = dict(B=2, T=5, D=8, K=4, x=at(0), ld=8, t=0, w=at(1), bias=at(2), wt=1, silu=1, state=at(3), lengths=None, dy=at(4), ld_dy=8,
             dlast=None, dx=at(5), dw=at(6), dbias=at(7), dstate=at(8), ws=at(9), n=1 << 20)
    a.update(kw)
    return lib.causal_conv_backward(*a.values(), None)


def conv_step(**kw):
    a = dict(B=2, D=8, K=4, x=at(0), ld=8, t=0, w=at(1), bias=at(2), wt=1, silu=1, state=at(3), next=at(3), y=at(4))
    a.update(kw)
    return lib.causal_conv_step(*a.values(), None)


CONV = [(dict(B=-1), BAD), (dict(D=-1), BAD), (dict(K=0), BAD), (dict(K=9), UNSUP), (dict(x=None), BAD), (dict(w=None), BAD),
        (dict(ld=7), BAD), (dict(ld=1 << 62), BAD), (dict(t=2), BAD), (dict(wt=-1), BAD), (dict(silu=2), BAD), (dict(x=at(0, 2)), BAD),
        (dict(w=at(1, 1)), BAD), (dict(bias=at(2, 1)), BAD), (dict(state=at(3, 2)), BAD), (dict(D=1 << 41), BAD)]


@pytest.mark.parametrize("kw,code", CONV + [
    (dict(T=-1), BAD), (dict(y=None), BAD), (dict(y=at(0)), BAD), (dict(y=at(1)), BAD), (dict(last=at(3)), BAD), (dict(last=at(4)), BAD),
    (dict(lengths=at(9, 2)), BAD), (dict(B=1 << 34, T=1), UNSUP)])
def test_conv_refusals(kw, code):
    assert conv(**kw) == code
    assert lib.scanrnn_last_error()


@pytest.mark.parametrize("kw,code", CONV + [
    (dict(T=-1), BAD), (dict(dy=None), BAD), (dict(dx=None), BAD), (dict(dw=None), BAD), (dict(ld_dy=7), BAD), (dict(dx=at(0)), BAD),
    (dict(dx=at(4)), BAD), (dict(dw=at(7)), BAD), (dict(dstate=at(3)), BAD), (dict(dw=at(6, 2)), BAD), (dict(ws=None), BAD),
    (dict(n=16), SMALL)])
def test_conv_backward_refusals(kw, code):
    assert conv_backward(**kw) == code
    assert lib.scanrnn_last_error()


@pytest.mark.parametrize("kw,code", CONV + [(dict(y=None), BAD), (dict(next=None), BAD), (dict(next=at(3, 4)), BAD), (dict(y=at(3)), BAD),
                                            (dict(next=at(0), state=None), BAD)])
def test_conv_step_refusals(kw, code):
    assert conv_step(**kw) == code
    assert lib.scanrnn_last_error()


def norm(**kw):
    a = dict(M=4, D=8, x=at(0), ld=8, t=1, r=at(1), ld_r=8, rt=0, w=at(2), wt=0, eps=1e-6, total=at(3), y=at(4))
    a.update(kw)
    return lib.rms_norm_forward(*a.values(), None)


def codes(**kw):
    a = dict(M=4, D=8, x=at(0), ld=8, t=1, r=at(1), ld_r=8, rt=0, w=at(2), wt=0, eps=1e-6, total=at(3), q=at(4), scale=at(5))
    a.update(kw)
    return lib.rms_norm_quantize(*a.values(), None)


NORM = [(dict(M=-1), BAD), (dict(D=0), BAD), (dict(D=-1), BAD), (dict(D=16385, ld=1 << 15, ld_r=1 << 15), UNSUP), (dict(x=None), BAD),
        (dict(w=None), BAD), (dict(ld=7), BAD), (dict(ld_r=7), BAD), (dict(t=2), BAD), (dict(rt=3), BAD), (dict(wt=3), BAD),
        (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD), (dict(eps=float("inf")), BAD), (dict(total=None), BAD),
        (dict(r=None), BAD), (dict(x=at(0, 1)), BAD), (dict(total=at(3, 2)), BAD), (dict(total=at(0)), BAD),
        (dict(total=at(1), ld_r=9), BAD), (dict(total=at(1, 4)), BAD), (dict(M=1 << 41), BAD), (dict(ld=1 << 62), BAD)]


@pytest.mark.parametrize("kw,code", NORM + [(dict(y=None), BAD), (dict(y=at(0)), BAD), (dict(y=at(3)), BAD), (dict(y=at(4, 1)), BAD),
                                            (dict(y=at(2)), BAD)])
def test_norm_refusals(kw, code):
    assert norm(**kw) == code
    assert lib.scanrnn_last_error()


@pytest.mark.parametrize("kw,code", NORM + [(dict(q=None), BAD), (dict(scale=None), BAD), (dict(q=at(4, 8)), BAD),
                                            (dict(scale=at(5, 2)), BAD), (dict(scale=at(4, 16)), BAD), (dict(scale=at(0)), BAD),
                                            (dict(q=at(1)), BAD)])
def test_norm_codes_refusals(kw, code):
    assert codes(**kw) == code
    assert lib.scanrnn_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), BAD), (dict(D=0), BAD), (dict(D=20000, ld=20000, ld_dy=20000, ld_dt=20000), UNSUP), (dict(total=None), BAD),
    (dict(dy=None), BAD), (dict(dx=None), BAD), (dict(dw=None), BAD), (dict(ld=7), BAD), (dict(ld_dy=7), BAD), (dict(ld_dt=7), BAD),
    (dict(eps=-1.0), BAD), (dict(dx=at(0)), BAD), (dict(dx=at(3)), BAD), (dict(dw=at(5)), BAD), (dict(dw=at(1)), BAD), (dict(ws=None), BAD),
    (dict(n=16), SMALL), (dict(w=None), BAD), (dict(t=2), BAD)])
def test_norm_backward_refusals(kw, code):
    a = dict(M=40, D=8, total=at(0), ld=8, t=0, w=at(1), wt=0, eps=1e-6, dy=at(2), ld_dy=8, gt=1, dt=at(3), ld_dt=8, dx=at(5), dw=at(6),
             ws=at(7), n=1 << 20)
    a.update(kw)
    assert lib.rms_norm_backward(*a.values(), None) == code
    assert lib.scanrnn_last_error()


def test_python_binding_refuses():
    x, x3, w = torch.zeros(2, 8), torch.zeros(2, 3, 8), torch.zeros(8, 4)
    h = torch.zeros(2, 8, 4)
    for call in (lambda: sr.selective_scan_forward(x3, x3, w, h[:, :3], h[:, :3]),
                 lambda: sr.selective_scan_backward(x3, x3, w, h[:, :3], h[:, :3], x3), lambda: sr.selective_step(x, x, w, x, x),
                 lambda: sr.selective_scan(x3, x3, w, h[:, :3], h[:, :3]), lambda: sr.causal_conv_forward(x3, w),
                 lambda: sr.causal_conv_backward(x3, w, x3), lambda: sr.causal_conv_step(x, w), lambda: sr.causal_conv(x3, w),
                 lambda: sr.rms_norm_forward(x, x[0]), lambda: sr.rms_norm_quantize(x, x[0]), lambda: sr.rms_norm(x, x[0]),
                 lambda: sr.rms_norm_backward(x, x[0], x)):
        with pytest.raises((ValueError, TypeError)):
            call()
