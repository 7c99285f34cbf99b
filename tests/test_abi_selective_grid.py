"""More workgroups than one launch takes are refused, however the sizes are spread."""

import pytest

from tests.test_abi_layers import UNSUP, scan, scan_backward, step

WIDE = 1 << 33


@pytest.mark.parametrize("G", [1, 1 << 20, 1 << 32, WIDE])
def test_wide_rows(G):
    ld = dict(B=1, D=WIDE, N=1, G=G, ld_u=WIDE, ld_d=WIDE, ld_z=WIDE, ld_b=G, ld_c=G)
    apart = {k: v + (1 << 50) * i for i, (k, v) in enumerate(dict.fromkeys(
        ("u", "delta", "z", "Bm", "Cm", "A", "skip", "bias", "y"), 1 << 51).items())}
    assert scan(T=1, **ld, **apart, ws=None, n=0) == UNSUP
    assert step(**ld, **apart, prev=None, next=1 << 54) == UNSUP


def test_many_sequences():
    for T in (0, 1):
        assert scan(B=1 << 30, T=T, N=32, ld_b=64, ld_c=64) == UNSUP
    assert scan_backward(B=1 << 34, T=0, D=1, G=1, n=1 << 62) == UNSUP
