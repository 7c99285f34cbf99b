"""What MinGRUInt8.requantize takes over, and what it refuses."""

import pytest
import torch

from tests.gpu_util import say
from tests.test_gpu_int8_layer import _layer

pytestmark = pytest.mark.gpu

sr = pytest.importorskip("scan_linear_rnn_amd")


def test_requantize_takes_over_the_decay():
    say("int8 layer requantize decay")
    x = torch.randn(3, 7, 16, device="cuda")
    gaps = torch.rand(3, 7, device="cuda") * 3
    q = _layer(decay_rate=0.1).quantized()
    for other in (_layer(decay_rate=0.7), _layer(decay_rate=0.7, log1p_delta=True), _layer(),
                  _layer(decay_rate=torch.linspace(0, 1, 16))):
        q.requantize(other)
        assert torch.equal(q(x, delta_t=gaps), other.quantized()(x, delta_t=gaps))


def test_requantize_refuses_another_shape_before_it_writes():
    say("int8 layer requantize refusals")
    layers = {"with": _layer(), "narrow": _layer(W_out=torch.randn(16, 8)), "without": _layer(W_out=False), "wide": _layer(expansion=2.0), "other": _layer(24)}
    for mine, other in (("with", "without"), ("without", "with"), ("with", "wide"), ("with", "other"),
                        ("without", "wide"), ("with", "narrow"), ("narrow", "with")):
        q = layers[mine].quantized()
        held = [t.clone() for t in (q.W_in, q.W_in_scale, q.W_out, q.W_out_scale) if t is not None]
        changed = layers[other]
        with pytest.raises(ValueError):
            q.requantize(changed)
        now = [t for t in (q.W_in, q.W_in_scale, q.W_out, q.W_out_scale) if t is not None]
        assert all(torch.equal(a, b) for a, b in zip(held, now))
    q = layers["without"].quantized()
    double = _layer(W_out=False)
    double.W_in.mul_(2)
    q.requantize(double)
    assert torch.equal(q.W_in_scale, sr.quantize_columns(double.W_in)[1])
