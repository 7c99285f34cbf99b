"""More threads than one launch takes are refused, however the sizes are spread."""

from tests.test_abi_layers import UNSUP, conv, conv_backward, conv_step


def test_wide_rows_and_many_sequences():
    D = 1 << 36
    far = {k: 1 << (50 + i) for i, k in enumerate(("x", "w", "bias", "y"))}
    kept = dict(state=None, last=None)
    assert conv(B=1, T=1, D=D, K=1, ld=D, **far, **kept) == UNSUP
    assert conv(B=1 << 34, T=0) == UNSUP
    for T in (0, 1):
        assert conv_backward(B=1 << 34, T=T, n=1 << 62) == UNSUP
    assert conv_step(B=1, D=D, K=1, ld=D, **far, state=None, next=None) == UNSUP
