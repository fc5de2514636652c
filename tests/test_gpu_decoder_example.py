"""The example's layer as a layer: its norms, and what it keeps between steps."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_expert_weight_gb300 import build
    build.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import decoder_layer
    decoder_layer.S.load()
    decoder_layer.S.device_status()
    return decoder_layer


@pytest.fixture(scope="module")
def layer(ex):
    return ex.DecoderLayer(ex.Y.WORKLOADS["tiny"], 8, 2, 64, torch.device(DEV))


def one_step(ex, layer, x):
    T = x.shape[0]
    cache = ex.PagedCache(8, 16, 2, 64, 1, 8, torch.device(DEV))
    return layer(x, cache, cache.grow([T]), T)


def test_what_a_layer_adds_does_not_grow_with_its_input(ex, layer):
    """Both halves norm their input, so 1,024 times the input changes the sum by the same
    order as the input itself: about 1 in 1,024, beside a rounding to bf16 (2^-8)."""
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    x = torch.randn(50, layer.wl.d, generator=g, device=DEV).bfloat16()
    y = one_step(ex, layer, x * 1024).double() / 1024
    added = (one_step(ex, layer, x).double() - x.double()).abs().max()
    assert float((y - x.double()).abs().max()) <= float(x.abs().max()) * 2.0 ** -7 + 4 * added / 1024
    assert ex.S.device_status() == 0


def test_few_workspaces_serve_every_number_of_rows(ex, layer):
    """Steps of 1 to 40 rows keep at most a workspace per power of two, and a row's output
    does not depend on what fills the rows up."""
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    x = torch.randn(40, layer.wl.d, generator=g, device=DEV).bfloat16()
    layer.moe_ws.clear()
    for T in range(1, 41):
        assert one_step(ex, layer, x[:T]).shape == (T, layer.wl.d)
    assert len(layer.moe_ws) <= 7
    whole = ex.S.forward(layer.experts, x[:8], ex.S.workspace(layer.experts, 8))
    assert torch.equal(layer.moe(x[:8]), whole)
    part = layer.moe(x[:5])
    assert bool(((part - whole[:5]).abs() <= 1e-4 * whole.abs().max()).all())
    assert ex.S.device_status() == 0
