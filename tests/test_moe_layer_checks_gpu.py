"""The 8-bit layer of examples/moe_layer.py refuses what its buffers were not
made for, before a kernel sees an address, and is whole at its own limits."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
N, K, D, FF = 16, 4, 512, 256


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


@pytest.fixture(scope="module")
def weights(ex):
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return (r(N, D) / D ** 0.5).to(torch.bfloat16).view(torch.int16), r(N, 2 * FF, D) / D ** 0.5, r(N, D, FF) / FF ** 0.5


def _x(T):
    return torch.randn(T, D, generator=torch.Generator(device="cuda").manual_seed(T + 1), device="cuda")


def _out(T):
    return torch.full((T, D), -7.0, dtype=torch.bfloat16, device="cuda")


@pytest.mark.parametrize("most,T", [(8, 9), (8, 32), (8, 300), (70, 71)])
def test_more_tokens_than_the_layer_was_made_for(ex, weights, most, T):
    layer, out = ex.Q8Layer(*weights, K, most), _out(T)
    with pytest.raises(ValueError, match="made for"):
        layer(_x(T), out)
    torch.cuda.synchronize()
    assert (out == -7).all()


@pytest.mark.parametrize("most", [8, 70])
def test_as_many_tokens_as_it_was_made_for(ex, weights, most):
    """Equal to the output of a layer made for more."""
    a, b = _out(most), _out(most)
    ex.Q8Layer(*weights, K, most)(_x(most), a)
    ex.Q8Layer(*weights, K, 4 * most)(_x(most), b)
    assert torch.equal(a, b) and not torch.isnan(a).any()
    assert ex.smoe.smoe_last_device_status() == ex.smoe.SMOE_OK


def test_arguments_of_the_call(ex, weights):
    layer, T = ex.Q8Layer(*weights, K, 8), 4
    wide = torch.zeros(T, 2 * D, device="cuda")
    for x, out in ((_x(T).to(torch.bfloat16), _out(T)), (_x(T).double(), _out(T)), (_x(T)[:, :-16].contiguous(), _out(T)),
                   (_x(T).flatten(), _out(T)), (wide[:, ::2], _out(T)), (wide[:, :D], _out(T)), (_x(T).cpu(), _out(T)),
                   (_x(T), _out(T).float()), (_x(T), _out(T - 1)), (_x(T), _out(D)[:, :T].t()), (_x(T), _out(T).cpu())):
        with pytest.raises((TypeError, ValueError)):
            layer(x, out)


def test_arguments_of_the_layer(ex, weights):
    gate, gate_up, down = weights
    for bad in ((gate.float(), gate_up, down), (gate[:-1], gate_up, down), (gate, gate_up[:-1], down), (gate, gate_up[:, :-2], down),
                (gate, gate_up, down[:, :, :-16]), (gate, gate_up, down[:, :-16]), (gate, gate_up.half(), down),
                (gate.cpu(), gate_up, down), (gate, gate_up.cpu(), down)):
        with pytest.raises((TypeError, ValueError)):
            ex.Q8Layer(*bad, K, 8)
    for w in (gate_up.cpu(), gate_up.half()):
        with pytest.raises((TypeError, ValueError)):
            ex.quantize_weights(w)


def test_a_strided_gate(ex, weights):
    gate, gate_up, down = weights
    wide = torch.zeros(N, 2 * D, dtype=torch.int16, device="cuda")
    wide[:, ::2] = gate
    a, b = _out(8), _out(8)
    ex.Q8Layer(gate, gate_up, down, K, 8)(_x(8), a)
    ex.Q8Layer(wide[:, ::2], gate_up, down, K, 8)(_x(8), b)
    assert torch.equal(a, b)


def test_no_tokens(ex, weights):
    layer = ex.Q8Layer(*weights, K, 8)
    out = _out(0)
    assert layer(_x(0), out) is out
    assert ex.smoe.smoe_last_device_status() == ex.smoe.SMOE_OK
