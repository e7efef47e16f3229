"""The many-token calls together, as examples/moe_layer.py uses them: the 8-bit
layer against a float64 form that quantises at the same places, the training
path's gradients against a float64 autograd of the plain layer."""
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


def _weights(n, d, d_ff, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return r(n, d) / d ** 0.5, r(n, 2 * d_ff, d) / d ** 0.5, r(n, d, d_ff) / d_ff ** 0.5, g


def _q(v):
    top = v.abs().amax(-1, keepdim=True)
    return torch.round(v * (127 / top)), top / 127


@pytest.mark.parametrize("T", [1, 7, 64, 300])
def test_q8_layer(ex, T):
    n, k, d, d_ff = 16, 4, 512, 256
    router, gate_up, down, g = _weights(n, d, d_ff, 1)
    router = router.to(torch.bfloat16)
    x = torch.randn(T, d, generator=g, device="cuda")
    layer = ex.Q8Layer(router.view(torch.int16), gate_up, down, k, 300)
    out = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    layer(x, out)
    assert ex.smoe.smoe_last_device_status() == ex.smoe.SMOE_OK
    # the layer's own selection (its logits are f32), then float64 with the same quantisation points
    idx, w = layer.idx[:T].long(), layer.w[:T].double()
    xq, xs = _q(x.double())
    gq, gs = _q(gate_up.double())
    dq, ds = _q(down.double())
    ref = torch.zeros(T, d, dtype=torch.float64, device="cuda")
    mag = torch.zeros(T, 1, dtype=torch.float64, device="cuda")
    for s in range(k):
        for t in range(T):
            e = idx[t, s]
            h = (gq[e] @ xq[t]) * xs[t] * gs[e].squeeze(-1)
            v = torch.nn.functional.silu(h[:d_ff]) * h[d_ff:]
            hq, hs = _q(v)
            y = (dq[e] @ hq) * hs * ds[e].squeeze(-1)
            ref[t] += w[t, s] * y
            # what moves a code by one step of 127: the f32 reciprocals, and h's bf16 (2^-8 of each value, and
            # SiLU's slope of at most 1.1); each moves hidden by at most 3 2^-8 of its largest value in one column
            step = 3 * 2.0 ** -8 * v.abs().amax() + hs.squeeze()
            mag[t] += w[t, s] * (step * (down[e].double().square().sum(1).amax().sqrt()) * 4 + 2.0 ** -8 * y.abs().amax() * 2)
    # independent errors of the d_ff columns: four standard deviations of sqrt(sum down^2) times one column's
    assert ((out.double() - ref).abs() <= mag).all()


def test_q8_layer_in_a_graph(ex):
    n, k, d, d_ff, T = 16, 4, 512, 256, 40
    router, gate_up, down, g = _weights(n, d, d_ff, 2)
    layer = ex.Q8Layer(router.to(torch.bfloat16).view(torch.int16), gate_up, down, k, T)
    x = torch.randn(T, d, generator=g, device="cuda")
    out, eager = (torch.empty(T, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    layer(x, out, s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        layer(x, out, s)
    for _ in range(3):
        x.copy_(torch.randn(T, d, generator=g, device="cuda"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        layer(x, eager)
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


@pytest.mark.parametrize("T,n,k", [(5, 4, 2), (33, 8, 3)])
def test_training_gradients(ex, T, n, k):
    d, d_ff = 48, 40
    router, gate_up, down, g = _weights(n, d, d_ff, 3)
    x = torch.randn(T, d, generator=g, device="cuda")
    target = torch.randn(T, d, generator=g, device="cuda")
    p32 = [p.clone().requires_grad_() for p in (x, router, gate_up, down)]
    out = ex.moe_train(*p32, k)
    ((out - target) ** 2).sum().backward()
    p64 = [p.double().clone().requires_grad_() for p in (x, router, gate_up, down)]
    x6, r6, gu6, dn6 = p64
    l = x6 @ r6.t()
    v, i = torch.sort(l, dim=1, descending=True, stable=True)
    w = torch.softmax(v[:, :k], 1)
    h = torch.einsum("td,tkfd->tkf", x6, gu6[i[:, :k]])
    a = torch.nn.functional.silu(h[..., :d_ff]) * h[..., d_ff:]
    y = torch.einsum("tkf,tkdf->tkd", a, dn6[i[:, :k]])
    ref = (w[..., None] * y).sum(1)
    ((ref - target.double()) ** 2).sum().backward()
    assert (v[:, k - 1] - v[:, k]).min() > 1e-5  # the selection is the same in f32
    assert torch.allclose(out.double(), ref, rtol=1e-4, atol=1e-5)
    for a, b in zip(p32, p64):
        # f32 sums of at most T k d terms: 1e-4 of the gradient's own size
        assert (a.grad.double() - b.grad).norm() <= 1e-4 * b.grad.norm()


def test_example_runs(ex, capsys):
    ex.main()
    assert "gradient norms" in capsys.readouterr().out
