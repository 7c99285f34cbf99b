"""The step with time decay where a workgroup goes through several tiles of
128 x 128: rates and gaps are loaded again for each tile while the next one's
operands are on their way.  Tolerances as in test_gpu_i8.py."""

import numpy as np
import pytest
import torch

from tests.gpu_util import dev, say
from tests.test_gpu_i8 import _activations, _gates, _h_close, _host, _layer

pytestmark = pytest.mark.gpu

sr = pytest.importorskip("scan_linear_rnn_amd")


@pytest.mark.parametrize("B,D_in,D_h", [(4100, 130, 1100), (9000, 100, 1025)])
@pytest.mark.parametrize("decay", [False, True])
def test_rows_of_a_step_of_many_tiles_equal_those_of_small_ones(B, D_in, D_h, decay):
    say(f"i8 persistent step B={B} {D_in}->{D_h} decay={decay}")
    assert -(-B // 128) * -(-2 * D_h // 128) > 512           # more tiles than workgroups
    rng = np.random.default_rng([3300, B, D_in, D_h])
    W_in, _ = _layer(rng, D_in, D_h, 0)
    wi = sr.quantize_columns(dev(W_in))
    x = dev(_activations(rng, B, D_in))
    h0 = dev(rng.standard_normal((B, D_h)).astype(np.float32))
    rate = dev(rng.uniform(0, 0.5, D_h).astype(np.float32))
    gap = dev(rng.exponential(2.0, B).astype(np.float32))

    def step(rows, **more):
        kw = dict(decay_rate=rate, delta_t=gap[rows]) if decay else {}
        return sr.mingru_step_i8(x[rows], *wi, h_prev=h0[rows], **kw, **more)[0]

    h = step(slice(None))
    for at in range(0, B - 512, 512):
        assert torch.equal(h[at:at + 37], step(slice(at, at + 37)))
    assert torch.equal(h[B - 37:], step(slice(B - 37, B)))
    _h_close(h, *_gates(_host(x), W_in, D_h), _host(h0),
             np.exp(-_host(rate)[None, :].astype(np.float64) * _host(gap)[:, None]) if decay else 1.0)
    for _ in range(3):                                       # and in place
        state = h0.clone()
        kw = dict(decay_rate=rate, delta_t=gap) if decay else {}
        sr.mingru_step_i8(x, *wi, h_prev=state, h_next=state, **kw)
        assert torch.equal(state, h)
