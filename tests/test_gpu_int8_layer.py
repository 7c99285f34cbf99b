"""MinGRUInt8 as the layer it was made from: its saturation warning."""

import warnings

import pytest
import torch

from tests.gpu_util import say

pytestmark = pytest.mark.gpu

sr = pytest.importorskip("scan_linear_rnn_amd")


def _layer(dim=16, **kw):
    g = torch.Generator()
    g.manual_seed(5000)
    return sr.MinGRU(dim, generator=g, **kw)


def _warnings_of(call):
    with warnings.catch_warnings(record=True) as caught:
        warnings.simplefilter("always")
        call()
    return [w for w in caught if issubclass(w.category, UserWarning)]


@pytest.mark.parametrize("token", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_saturation_warning(token, dtype):
    say(f"int8 layer warning token={token} {dtype}")
    x = torch.randn(2, 16, device="cuda", dtype=dtype) if token else torch.randn(2, 5, 16, device="cuda", dtype=dtype)
    small, large = torch.ones(x.shape[:-1], device="cuda"), torch.full(x.shape[:-1], 1e6, device="cuda")
    q = _layer(decay_rate=0.5).quantized()
    assert not _warnings_of(lambda: q(x))
    assert not _warnings_of(lambda: q(x, delta_t=small))
    caught = _warnings_of(lambda: q(x, delta_t=large))
    assert len(caught) == 1 and str(caught[0].message) == sr.MinGRU.SATURATION_WARNING
    assert caught[0].filename == __file__                            # of the caller's line
    assert not _warnings_of(lambda: q(x, delta_t=large))             # once per layer
    silent = _layer(decay_rate=0.5, warn_saturation=False).quantized()
    assert not _warnings_of(lambda: silent(x, delta_t=large))
    logs = _layer(decay_rate=0.5, log1p_delta=True).quantized()
    assert not _warnings_of(lambda: logs(x, delta_t=large))


def test_the_warning_does_not_change_the_result():
    say("int8 layer warning result")
    x = torch.randn(3, 7, 16, device="cuda")
    gaps = torch.rand(3, 7, device="cuda") * 1e5
    a, b = (_layer(decay_rate=0.5, warn_saturation=on).quantized() for on in (True, False))
    with warnings.catch_warnings():
        warnings.simplefilter("ignore")
        assert torch.equal(a(x, delta_t=gaps), b(x, delta_t=gaps))


def test_a_decayed_layer_is_recorded_into_a_graph():
    """Nothing is read while a graph is recorded: the warning waits for the
    next call outside of it."""
    say("int8 layer warning graph")
    layer = _layer(decay_rate=0.5)
    q = layer.quantized()
    x, h = torch.randn(3, 16, device="cuda"), torch.randn(3, 16, device="cuda")
    gaps = torch.full((3,), 1e6, device="cuda")
    ref = q(x, h)                                            # no decay: a warm-up
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q(x, h, delta_t=torch.ones(3, device="cuda"))
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = q(x, h, delta_t=gaps)
    for _ in range(3):
        q(x, h)
        torch.cuda.synchronize()
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, _layer(decay_rate=0.5, warn_saturation=False).quantized()(x, h, delta_t=gaps))
        assert not torch.equal(y, ref)
    assert len(_warnings_of(lambda: q(x, h, delta_t=torch.ones(3, device="cuda")))) == 1
