"""The library has first gradients only: a second one through its calls is
refused, where it used to come back without their terms."""
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


@pytest.mark.parametrize("which", ["top_k", "dispatch", "combine"])
def test_a_second_gradient_is_refused(ex, which):
    T, n, k, d = 6, 8, 2, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    l, x, ys, w = r(T, n).requires_grad_(), r(T, d).requires_grad_(), r(T * k, d).requires_grad_(), r(T, k).requires_grad_()
    idx, _ = ex.top_k(l.detach(), k)
    _, _, place = ex.dispatch(x.detach(), idx, n)
    out, arg = {"top_k": lambda: (ex.top_k(l, k)[1], l), "dispatch": lambda: (ex.dispatch(x, idx, n)[0], x),
                "combine": lambda: (ex.combine(ys, place, w), w)}[which]()
    first, = torch.autograd.grad(out.square().sum(), arg, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        first.square().sum().backward()
