"""The limit on the distance of the selective scan's rows goes by what is addressed
with it: one token has none (a call of no sequences shows it without a launch)."""

import pytest

from tests.test_abi_layers import OK, UNSUP, scan, scan_backward


@pytest.mark.parametrize("ld", ["ld_u", "ld_d", "ld_z", "ld_b", "ld_c"])
def test_distance_of_rows(ld):
    assert scan(B=0, T=1, **{ld: 1 << 26}) == OK
    assert scan(B=0, T=0, **{ld: 1 << 26}) == OK
    assert scan(T=2, **{ld: 1 << 26}) == UNSUP
    assert scan_backward(T=2, **{ld: 1 << 26}) == UNSUP
