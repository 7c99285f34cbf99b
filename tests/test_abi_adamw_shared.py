"""AdamW refuses two tensors of a step that share memory: their workgroups
would update it at the same time.  Checked before anything is launched."""

import pytest

from tests.test_abi_adamw_each import _each
from tests.test_abi_i8 import BAD, UNSUP, _adamw

sr = pytest.importorskip("scan_linear_rnn_amd")
lib = sr.raw_library()

G = 0x9000000


@pytest.mark.parametrize("tensors", [
    ((0x10000, G, 4, 0, 0), (0x10000, G, 4, 0, 0)),                                # the same twice
    ((0x10000, G, 4, 0, 0), (0x20000, G, 4, 0, 0), (0x10000, G, 4, 0, 0)),
    ((0x10000, G, 100, 0, 0), (0x10000 + 396, G, 4, 0, 0)),                        # one element, fp32
    ((0x10000 + 198, G, 4, 1, 0), (0x10000, G, 100, 1, 0)),                        # bf16, the other order
    ((0x10000, G, 4096, 0, 0), (0x10100, G, 1, 1, 0), (0x80000, G, 1, 0, 0)),      # inside
    tuple((0x100000 + 64 * (i * 37 % 400), G, 16, 0, 0) for i in range(400)) + ((0x100000 + 64 * 133 + 4, G, 1, 0, 0),)])
def test_tensors_that_share_memory(tensors):
    n = sum(-(-t[2] // 256) * 256 for t in tensors)
    assert _adamw(tensors=tensors, n=n) == BAD
    assert b"share memory" in lib.scanrnn_last_error()
    assert _each(tensors=tensors, steps=tuple(range(1, 1 + len(tensors))), n=n) == BAD
    assert b"share memory" in lib.scanrnn_last_error()


def test_the_grid_limit_comes_first():
    assert _adamw(tensors=((0x10000, G, 1 << 40, 0, 0), (0x10000, G, 4, 0, 0)), n=1 << 41) == UNSUP


def test_tensors_that_do_not_take_part_may_share():
    assert _adamw(tensors=((0x10000, 0, 4, 0, 0), (0x10000, 0, 4, 0, 0), (0x10000, G, 0, 0, 0))) == sr.SR_OK
