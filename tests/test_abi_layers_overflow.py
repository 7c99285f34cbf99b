"""Sizes near 2^63 in the layer operators' calls are refused without computing with
them (the sanitizers' copy of the library reports an overflow)."""

import pytest

from tests.test_abi_layers import BAD, codes, conv, conv_backward, conv_step, lib, norm, scan, scan_backward, step

MOST = (1 << 63) - 1


@pytest.mark.parametrize("v", [MOST, MOST - 100])
def test_sizes_near_the_largest_integer(v):
    for call, names in ((conv, "BTD"), (conv_backward, "BTD"), (conv_step, "BD"), (scan, "BTD"), (scan_backward, "BTD"), (step, "BD")):
        for name in names:
            assert call(**{name: v}) == BAD, (call, name)
    for call in (norm, codes):
        for kw in (dict(D=v), dict(M=v), dict(M=0, D=v), dict(D=v, ld=v, ld_r=v)):
            assert call(**kw) == BAD, (call, kw)
    for T in (v, 1 << 62):
        assert lib.causal_conv_backward_workspace_size(1, T, 8, 4, 0) == 0
        assert lib.selective_scan_backward_workspace_size(1, T, 8, 4, 1) == lib.selective_scan_forward_workspace_size(1, T, 8, 4, 1) == 0
    assert lib.rms_norm_backward_workspace_size(v, 8) == lib.rms_norm_backward_workspace_size(8, v) == 0


@pytest.mark.parametrize("v", [MOST, MOST - 100])
def test_norm_backward_sizes(v):
    from tests.test_abi_layers import at
    for M, D, ld in ((4, v, v), (0, v, v), (v, 8, 8)):
        assert lib.rms_norm_backward(M, D, at(0), ld, 0, at(1), 0, 1e-6, at(2), ld, 1, at(3), ld, at(5), at(6), at(7), 1 << 20, None) == BAD
