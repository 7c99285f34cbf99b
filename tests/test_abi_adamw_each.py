"""Refusals of adamw_step_each: every check runs before anything is launched."""

import ctypes

import pytest

from tests.test_abi_i8 import A, B, BAD, C, D, ODD

sr = pytest.importorskip("scan_linear_rnn_amd")
lib = sr.raw_library()

TENSORS = ((0x10000, 0x20000, 4, 0, 0), (0x30000, 0x40000, 4, 0, 0))


def _each(tensors=TENSORS, steps=(1, 1), m=A, v=B, ms=None, vs=None, bits=32, n=1024, lr=1e-3, b1=0.9, b2=0.99,
          eps=1e-8, wd=0.0, gs=None):
    flat = [x for p, g, k, pt, gt in tensors for x in (p, g, k, (pt & 0xFFFFFFFF) | gt << 32)]
    table = (ctypes.c_int64 * len(flat))(*flat) if flat else None
    numbers = (ctypes.c_int64 * len(steps))(*steps) if steps else None
    return lib.adamw_step_each(len(tensors), table, m, v, ms, vs, bits, n, numbers, lr, b1, b2, eps, wd, gs, None)


@pytest.mark.parametrize("kw", [
    dict(steps=None), dict(steps=(1, 0)), dict(steps=(-3, 1)), dict(bits=16), dict(b1=1.0), dict(lr=float("nan")),
    dict(m=None), dict(v=ODD), dict(n=256), dict(ms=C, vs=D), dict(bits=8), dict(gs=ctypes.c_void_p(0x10001)),
    dict(tensors=((0, 0x20000, 4, 0, 0),), steps=(1,)), dict(tensors=((0x10000, 0x20000, 4, 3, 0),), steps=(1,))])
def test_refusals(kw):
    assert _each(**kw) == BAD
    assert lib.scanrnn_last_error()


def test_calls_without_work_launch_nothing():
    assert _each(tensors=(), steps=None) == sr.SR_OK
    # Without a gradient a tensor's step number is not read.
    assert _each(tensors=((0x10000, 0, 4, 0, 0),), steps=(0,)) == sr.SR_OK
