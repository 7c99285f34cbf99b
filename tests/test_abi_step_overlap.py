"""mingru_step_i8 refuses a new state that overlaps what the step still reads:
its workgroups write states while others read.  Checked before any launch."""

import ctypes

import pytest

from tests.test_abi_i8 import BAD, _step

sr = pytest.importorskip("scan_linear_rnn_amd")
lib = sr.raw_library()


def P(n):
    return ctypes.c_void_p(n)


# B = 2, D_in = D_h = D_out = 4: x_t 32 bytes of fp32 or 16 of bf16, states 32 bytes.
@pytest.mark.parametrize("kw,which", [
    (dict(x=P(0x50000), hn=P(0x50000)), b"x_t"),
    (dict(x=P(0x50000), hn=P(0x50000 + 28)), b"x_t"),
    (dict(x=P(0x50000 + 28), hn=P(0x50000)), b"x_t"),
    (dict(x=P(0x50000), t=1, hn=P(0x50000 + 12)), b"x_t"),
    (dict(x=P(0x50000), hn=P(0x50000), hp=P(0x50000)), b"x_t"),
    (dict(hp=P(0x50000), hn=P(0x50000 + 4)), b"h_prev"),
    (dict(hp=P(0x50000 + 16), hn=P(0x50000)), b"h_prev"),
    (dict(wo=P(0x20000), so=P(0x30000), hn=P(0x50000), y=P(0x50000)), b"y_t"),
    (dict(wo=P(0x20000), so=P(0x30000), hn=P(0x50000), y=P(0x50000 + 28)), b"y_t"),
    (dict(wo=P(0x20000), so=P(0x30000), t=1, hn=P(0x50000 + 12), y=P(0x50000)), b"y_t"),
])
def test_a_state_that_overlaps(kw, which):
    assert _step(**kw) == BAD
    assert b"overlap" in lib.scanrnn_last_error() and which in lib.scanrnn_last_error()
