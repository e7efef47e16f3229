"""The 8-bit layer of examples/moe_layer.py over any number of experts: the
logits of a token begin wherever the row before them ends."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U = 2.0 ** -24


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


@pytest.mark.parametrize("n", [3, 6, 9, 12])
@pytest.mark.parametrize("T", [1, 5, 70])
def test_number_of_experts(ex, n, T):
    k, d, d_ff = 2, 64, 32
    g = torch.Generator(device="cuda").manual_seed(n)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    gate = (r(n, d) / d ** 0.5).to(torch.bfloat16)
    layer = ex.Q8Layer(gate.view(torch.int16), r(n, 2 * d_ff, d) / d ** 0.5, r(n, d, d_ff) / d_ff ** 0.5, k, 70)
    x, out = r(T, d), torch.full((T, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    layer(x, out)
    assert ex.smoe.smoe_last_device_status() == ex.smoe.SMOE_OK
    assert torch.isfinite(out).all()
    logits = layer.logits[:T]
    x64, g64 = x.double(), gate.double()
    assert ((logits.double() - x64 @ g64.t()).abs() <= (d + 1) * U * (x64.abs() @ g64.abs().t())).all()
    assert torch.equal(layer.idx[:T].long(), torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k])
