"""One token of each sequence, taken out of a buffer whose sequences are far apart: the
distance of the rows is then a whole sequence's, which no offset within a tile
depends on."""

import pytest
import torch

from tests.gpu_util import say
from tests.test_gpu_selective import GRADS, args, case, given

pytestmark = pytest.mark.gpu

sr = pytest.importorskip("scan_linear_rnn_amd")


@pytest.mark.parametrize("apart,B,lengths", [(1 << 26, 3, None), (1 << 26, 3, [1, 0, 1]), ((1 << 31) + 8, 2, None)])
def test_one_token_of_long_sequences(apart, B, lengths):
    say("selective scan, one token of sequences", apart, "elements apart")
    D, N, at = 130, 16, 5
    c = case(B, 1, D, N, dtype="bf16", lengths=lengths)
    far = torch.empty((B - 1) * apart + 1024, dtype=torch.bfloat16, device="cuda")
    v = dict(c)
    for name in ("u", "delta", "z", "B", "C", "dy"):
        flat = c[name].reshape(B, 1, -1)
        part = far.as_strided((B, 1, flat.shape[2]), (apart, flat.shape[2], 1), at)
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
