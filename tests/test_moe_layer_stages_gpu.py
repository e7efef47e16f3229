"""The 8-bit layer of examples/moe_layer.py stage by stage: every stage's output
against float64 on the stage's own inputs as the layer left them on the
device, so that the bounds are those of its own rounding alone (u = 2^-24, 2^-8
for a bf16 output)."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U, BF = 2.0 ** -24, 2.0 ** -8


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


def _codes(v):
    """Codes and scales by their definition in f32."""
    top = v.abs().amax(-1, keepdim=True)
    return torch.round(v * (torch.full_like(top, 127.0) / top)).to(torch.int8), (top / torch.full_like(top, 127.0)).squeeze(-1)


def _product(q, s, wq, ws, expert):
    """Row r by expert[r]'s matrix; below 2^24 the integer sums are exact."""
    y = torch.empty(q.shape[0], wq.shape[1], dtype=torch.float64, device="cuda")
    for e in range(wq.shape[0]):
        r = expert == e
        y[r] = (q[r].double() @ wq[e].double().t()) * s[r].double()[:, None] * ws[e].double()
    return y


@pytest.mark.parametrize("T", [1, 7, 64, 65, 300])
def test_every_stage(ex, T):
    n, k, d, d_ff = 16, 4, 512, 256
    g = torch.Generator(device="cuda").manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    router, gate_up, down = (r(n, d) / d ** 0.5).to(torch.bfloat16), r(n, 2 * d_ff, d) / d ** 0.5, r(n, d, d_ff) / d_ff ** 0.5
    x = r(T, d)
    layer = ex.Q8Layer(router.view(torch.int16), gate_up, down, k, 300)
    out = torch.full((T, d), -7.0, dtype=torch.bfloat16, device="cuda")
    layer(x, out)
    assert ex.smoe.smoe_last_device_status() == ex.smoe.SMOE_OK
    R = T * k
    # the weights' codes
    for w, q, s in ((gate_up, layer.gu, layer.gu_scales), (down, layer.dn, layer.dn_scales)):
        wq, ws = _codes(w)
        assert torch.equal(q, wq) and torch.equal(s, ws)
    # the router: at most d roundings of each product and sum
    logits = layer.logits[:T]
    x64, r64 = x.double(), router.double()
    assert ((logits.double() - x64 @ r64.t()).abs() <= (d + 1) * U * (x64.abs() @ r64.abs().t())).all()
    # the selection of those logits
    v, i = torch.sort(logits, dim=1, descending=True, stable=True)
    idx, w = layer.idx[:T], layer.w[:T]
    assert torch.equal(idx.long(), i[:, :k])
    span = (v[:, :1] - v[:, k - 1:k]).double()
    ref = torch.softmax(v[:, :k].double(), 1)
    assert ((w.double() - ref).abs() <= U * (span + 16) * ref).all()
    # the sort
    order = torch.argsort(idx.flatten(), stable=True)
    assert torch.equal(layer.order[:R].long(), order)
    place = layer.place[:R].long()
    assert torch.equal(place[order], torch.arange(R, device="cuda"))
    expert = idx.flatten()[order]
    # the tokens' codes, the first product
    xq, xs = _codes(x)
    assert torch.equal(layer.xq[:T], xq) and torch.equal(layer.x_scales[:T], xs)
    h = layer.h[:R].double()
    ref = _product(xq[order // k], xs[order // k], layer.gu, layer.gu_scales, expert)
    assert ((h - ref).abs() <= (3 * U + BF) * ref.abs()).all()
    # the activation's codes: half a step and the roundings of 127 steps
    ref = torch.nn.functional.silu(h[:, :d_ff]) * h[:, d_ff:]
    step = ref.abs().amax(1, keepdim=True) / 127
    hq, hs = layer.hq[:R], layer.h_scales[:R]
    assert ((hs.double()[:, None] - step).abs() <= 12 * U * step).all()
    assert ((hq.double() * step - ref).abs() <= (0.5 + 127 * 26 * U) * step).all()
    # the second product, the sum
    ys = layer.ys[:R].double()
    ref = _product(hq, hs, layer.dn, layer.dn_scales, expert)
    assert ((ys - ref).abs() <= (3 * U + BF) * ref.abs()).all()
    prod = ys[place].view(T, k, d) * w.double()[..., None]
    ref = prod.sum(1)
    assert ((out.double() - ref).abs() <= U * (k + 1) * prod.abs().sum(1) + BF * ref.abs()).all()
