"""The routing of examples/moe_layer.py under autograd with the types that a
program hands it: logits that autocast made bf16, int64 indices, bf16 weights,
rows that a transpose left strided."""
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


def _r(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, device="cuda")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float64])
def test_logits_of_other_types(ex, dtype):
    """The selection is that of the values, the gradient comes in their type."""
    T, n, k = 33, 24, 4
    r = _r(1)
    l, d_w = r(T, n).to(dtype).requires_grad_(), r(T, k)
    idx, w = ex.top_k(l, k)
    v, i = torch.sort(l.detach().float(), dim=1, descending=True, stable=True)
    assert torch.equal(idx.long(), i[:, :k])
    assert torch.allclose(w.double(), torch.softmax(v[:, :k].double(), 1), rtol=U * 32, atol=0)
    (w * d_w).sum().backward()
    assert l.grad.dtype == dtype
    l32 = l.detach().float().requires_grad_()
    (ex.top_k(l32, k)[1] * d_w).sum().backward()
    assert torch.equal(l.grad, l32.grad.to(dtype))


@pytest.mark.parametrize("dtype", [torch.int64, torch.int32, torch.int16])
def test_indices_of_other_types(ex, dtype):
    T, n, k, d = 21, 16, 3, 40
    r = _r(2)
    idx = torch.sort(r(T, n), dim=1).indices[:, :k]
    idx[3, 1], idx[5, 0], idx[6, 2] = -1, n, -300
    if dtype == torch.int64:
        idx[7, 0], idx[8, 0] = (1 << 32) + 2, -(1 << 32) + 2  # no expert either
    there = (idx >= 0) & (idx < n)
    x = r(T, d)
    xs, offsets, place = ex.dispatch(x, idx.to(dtype), n)
    key = torch.where(there, idx, n).flatten()
    order = torch.argsort(key, stable=True)
    assert torch.equal(offsets.long(), torch.searchsorted(key[order], torch.arange(n + 1, device="cuda")))
    assert torch.equal(xs, torch.where(there.flatten()[order][:, None], x[order // k], 0.0))
    assert torch.equal(place >= 0, there.flatten())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float64])
def test_weights_of_other_types(ex, dtype):
    T, n, k, d = 19, 8, 2, 24
    r = _r(3)
    _, _, place = ex.dispatch(r(T, d), torch.sort(r(T, n), dim=1).indices[:, :k], n)
    ys, w = r(T * k, d).requires_grad_(), r(T, k).to(dtype).requires_grad_()
    out = ex.combine(ys, place, w)
    w32 = w.detach().float().requires_grad_()
    ref = ex.combine(ys, place, w32)
    assert torch.equal(out, ref)
    out.square().sum().backward()
    ys.grad = None
    ref.square().sum().backward()
    assert w.grad.dtype == dtype and torch.equal(w.grad, w32.grad.to(dtype))


def test_strided_arguments(ex):
    T, n, k, d = 12, 10, 3, 16
    r = _r(4)
    l, x = r(n, T).t(), r(d, T).t()
    idx, w = ex.top_k(l, k)
    idx_c, w_c = ex.top_k(l.contiguous(), k)
    assert torch.equal(idx, idx_c) and torch.equal(w, w_c)
    wide = torch.full((T, 2 * k), -1, device="cuda")
    wide[:, ::2] = idx.long()
    got, ref = ex.dispatch(x, wide[:, ::2], n), ex.dispatch(x.contiguous(), idx, n)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    twice = got[2].repeat_interleave(2)
    assert torch.equal(ex.combine(got[0], twice[::2], w), ex.combine(got[0], got[2], w))


@pytest.mark.parametrize("T,n,k", [(5, 4, 2), (40, 24, 3)])
def test_training_under_autocast(ex, T, n, k):
    """The router's product stays in f32, so that the selection is the one
    without autocast; the experts' products are bf16: three of them and an
    activation, whose roundings (2^-8 each, of sums of random signs) leave the output and
    the gradients within 2^-4 of their norm."""
    d, d_ff = 48, 40
    r = _r(5)
    params = r(T, d), r(n, d) / d ** 0.5, r(n, 2 * d_ff, d) / d ** 0.5, r(n, d, d_ff) / d_ff ** 0.5
    v = torch.sort(params[0].double() @ params[1].double().t(), dim=1, descending=True).values
    assert (v[:, k - 1] - v[:, k]).min() > 1e-5  # the selection is the same in f32
    target = r(T, d)
    grads = []
    for on in (False, True):
        p = [q.clone().requires_grad_() for q in params]
        with torch.autocast("cuda", torch.bfloat16, enabled=on):
            out = ex.moe_train(*p, k)
        ((out.float() - target) ** 2).sum().backward()
        grads.append([out.detach().float()] + [q.grad for q in p])
    for a, b in zip(*grads):
        assert (a - b).norm() <= 2.0 ** -4 * a.norm()
    assert ex.smoe.smoe_last_device_status() == ex.smoe.SMOE_OK


def test_refusals(ex):
    """What no conversion mends is refused before a kernel sees an address."""
    r = _r(6)
    T, n, k, d = 6, 8, 2, 16
    idx = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    w = torch.ones(T, k, device="cuda")
    xs, _, place = ex.dispatch(r(T, d), idx, n)
    for bad in (lambda: ex.top_k(r(T, n).cpu(), k), lambda: ex.top_k(r(T, n).int(), k), lambda: ex.top_k(r(n), k),
                lambda: ex.dispatch(r(T, d).cpu(), idx, n), lambda: ex.dispatch(r(T, d), idx.cpu(), n),
                lambda: ex.dispatch(r(T, d), idx.float(), n), lambda: ex.dispatch(r(T, d), idx[:-1], n),
                lambda: ex.dispatch(r(T, d).half(), idx, n), lambda: ex.dispatch(r(T, d), idx.flatten(), n),
                lambda: ex.combine(xs[:-1], place, w), lambda: ex.combine(xs, place[:-1], w), lambda: ex.combine(xs, place, w[:-1]),
                lambda: ex.combine(xs, place.long(), w), lambda: ex.combine(xs.half(), place, w), lambda: ex.combine(xs, place, w.cpu()),
                lambda: ex.combine(xs.cpu(), place, w), lambda: ex.combine(xs, place, w.int())):
        with pytest.raises((TypeError, ValueError)):
            bad()
