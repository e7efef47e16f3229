"""Sizes and parameters that a user's model has: those that the layers do not take are
refused in words, parameters that need a gradient are served."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build_library()
    spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def weights(n, d, ff):
    g = torch.Generator(device="cuda").manual_seed(n)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return (r(n, d) / d ** 0.5).to(torch.bfloat16), r(n, 2 * ff, d) / d ** 0.5, r(n, d, ff) / ff ** 0.5, r


@pytest.mark.parametrize("layer", ["Q8Layer", "F8Layer"])
@pytest.mark.parametrize("d,ff", [(72, 64), (64, 72), (100, 36), (64, 8)])
def test_sizes_that_are_no_multiples_of_16(ex, layer, d, ff):
    gate, gate_up, down, _ = weights(4, d, ff)
    with pytest.raises(ValueError, match="multiples of 16"):
        getattr(ex, layer)(gate, gate_up, down, 2, 8)


def test_sizes_that_the_library_refuses(ex):
    gate, gate_up, down, r = weights(4, 64, 32)
    with pytest.raises(ValueError, match="the library refuses"):
        ex.F8Layer(gate, gate_up, down, 65, 1)  # more slots a token than there are
    idx = torch.zeros(2, 65, dtype=torch.int32, device="cuda")
    with pytest.raises((ValueError, ex.smoe.SmoeError)):
        ex.dispatch(r(2, 64), idx, 4)


@pytest.mark.parametrize("layer", ["Q8Layer", "F8Layer"])
@pytest.mark.parametrize("T", [3, 70])
def test_parameters_and_rows_that_need_a_gradient(ex, layer, T):
    """A trained model's parameters as they are: served as their values are."""
    gate, gate_up, down, r = weights(8, 144, 80)
    x = r(T, 144)
    outs = []
    for own in (lambda t: t, torch.nn.Parameter):
        out = torch.full((T, 144), float("nan"), dtype=torch.bfloat16, device="cuda")
        served = getattr(ex, layer)(own(gate), own(gate_up), own(down), 2, 70)
        outs.append(served(own(x), out))
    assert torch.equal(*outs) and not outs[0].isnan().any() and not outs[1].requires_grad
    assert ex.smoe.smoe_last_device_status() == ex.smoe.SMOE_OK


def test_tensors_of_another_device_than_the_current_one(ex, monkeypatch):
    """The calls run on the current device's stream: refused before anything is launched."""
    gate, gate_up, down, r = weights(4, 64, 32)
    layer, out = ex.F8Layer(gate, gate_up, down, 2, 4), torch.full((3, 64), -7.0, dtype=torch.bfloat16, device="cuda")
    x, idx, offsets = r(3, 64), torch.zeros(3, 2, dtype=torch.int32, device="cuda"), torch.zeros(5, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    with monkeypatch.context() as m:
        m.setattr(torch.cuda, "current_device", lambda: 1)
        for call in (lambda: layer(x, out), lambda: ex.F8Layer(gate, gate_up, down, 2, 4), lambda: ex.route(r(3, 4), 2),
                     lambda: ex.top_k(r(3, 4), 2), lambda: ex.dispatch(x, idx, 4), lambda: ex.experts_f8(x, gate_up, offsets),
                     lambda: ex.combine(r(6, 64), torch.zeros(6, dtype=torch.int32, device="cuda"), r(3, 2)),
                     lambda: ex.quantize_weights(gate_up)):
            with pytest.raises(ValueError, match="current device"):
                call()
    torch.cuda.synchronize()
    assert (out == -7).all()
    layer(x, out)
    assert ex.smoe.smoe_last_device_status() == ex.smoe.SMOE_OK and (out != -7).any()
