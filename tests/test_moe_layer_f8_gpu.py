"""Scored routing, the 8-bit floating-point products and the weights' gradient
together, as examples/moe_layer.py uses them: every stage of a layer against
float64 of what that stage was given, the layer and a whole training step in a
CUDA graph, two streams at once."""
import importlib.util
import os

import numpy as np
import pytest

import f8_util as u

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U = 2.0 ** -24
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
N, K, D, FF = 16, 4, 512, 256
GROUPED = dict(score=1, n_groups=4, top_groups=2, group_best=2, norm=True, scale=2.5)


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


def _weights(seed, n=N, d=D, d_ff=FF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return (r(n, d) / d ** 0.5).to(torch.bfloat16), r(n, 2 * d_ff, d) / d ** 0.5, r(n, d, d_ff) / d_ff ** 0.5, r(n) / 8, r


def _f64(a):
    return torch.from_numpy(np.asarray(a)).cuda()


def _weights64(q, s):
    return _f64(u.weights_of(q.cpu().numpy(), s.cpu().numpy()))


def _rows64(q, s):
    return _f64(u.rows_of(q.cpu().numpy(), s.cpu().numpy()))


def _by_expert(x, w, offsets, rows=None):
    """(products, sums of magnitudes) of float64 rows and matrices; zeros behind the last."""
    at = offsets.tolist()
    y = torch.zeros(rows if rows is not None else x.shape[0], w.shape[1], dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(y)
    for e in range(w.shape[0]):
        y[at[e]:at[e + 1]] = x[at[e]:at[e + 1]] @ w[e].t()
        mag[at[e]:at[e + 1]] = x[at[e]:at[e + 1]].abs() @ w[e].abs().t()
    return y, mag


def _product_holds(got, ref, mag, n_in):
    """A block's 128 f32 sums (of the tensor core's own steps of 2^-23), a product by
    the scales and a sum for each block, one rounding to the type."""
    err = (128 + -(-n_in // 128) + 4) * 2.0 ** -23 * mag
    return ((got.double() - ref).abs() <= err + ROUND[got.dtype] * (ref.abs() + err) + 1e-37).all()


def _stages(ex, layer, x, out, bias, how):
    T, k, n, d, ff = x.shape[0], layer.k, layer.n, layer.d, layer.d_ff
    R = T * k
    logits, idx, w = layer.logits[:T], layer.idx[:T], layer.w[:T]
    x64, g64 = x.double(), layer.gate.double()
    # the products' sums of d terms in f32
    assert ((logits.double() - x64 @ g64.t()).abs() <= (d + 1) * U * (x64.abs() @ g64.abs().t())).all()
    l = logits.cpu().numpy()
    soft = how.get("score", 0) == 0
    ri = u.choose(l, None if bias is None else bias.cpu().numpy(), soft, how.get("n_groups", 1), how.get("top_groups", 1),
                  how.get("group_best", 1), k)
    assert (idx.cpu().numpy() == ri).all()
    rw = u.weights(l, ri, soft, how.get("norm", True), how.get("scale", 1.0))
    # exp and divide by 4 units at most, sums of n terms in 32 lanes, a divide
    assert (np.abs(w.cpu().numpy() - rw) <= (20 + n / 32 + 32) * 2 * U * np.abs(rw) + 1e-37).all()
    # the sorted order: every slot of an expert, in token order
    slots = ri.reshape(-1)
    order = layer.order[:R].cpu().numpy()
    at = layer.offsets.cpu().numpy()
    for e in range(n):
        assert (order[at[e]:at[e + 1]] == np.nonzero(slots == e)[0]).all()
    q, s = u.quantize_rows(x.cpu().numpy())
    assert (layer.xq[:T].cpu().numpy() == q).all() and (layer.x_scales[:T].cpu().numpy() == s).all()
    src = torch.from_numpy(order.astype(np.int64)).cuda() // k
    last = at[n]
    rows = torch.zeros(R, d, dtype=torch.float64, device="cuda")
    rows[:last] = _f64(u.rows_of(q, s))[src[:last]]
    h, hs, ys = layer.h[:R], layer.h_scales[:R], layer.ys[:R]
    assert _product_holds(h, *_by_expert(rows, _weights64(layer.gu, layer.gu_scales), layer.offsets), d)
    h64 = h.double()
    v = torch.nn.functional.silu(h64[:, :ff]) * h64[:, ff:]
    hidden = _rows64(layer.hq[:R], hs)
    spread = _f64(u.spread(hs.double().cpu().numpy(), 1, ff))
    # half a step of a code (2^-4 of it, or half of 2^-9 scales) and the activation in f32
    assert ((hidden - v).abs() <= (2.0 ** -4 + 2.0 ** -18) * v.abs() + spread * (2.0 ** -10 + 1e-6)).all()
    assert _product_holds(ys, *_by_expert(hidden, _weights64(layer.dn, layer.dn_scales), layer.offsets), ff)
    y64 = torch.zeros(R, d, dtype=torch.float64, device="cuda")
    for j in range(last):
        y64[order[j]] = ys[j].double()
    terms = y64.view(T, k, d) * w.double()[:, :, None]
    ref, mag = terms.sum(1), terms.abs().sum(1)
    assert ((out.double() - ref).abs() <= (k + 1) * U * mag + 2.0 ** -8 * (ref.abs() + (k + 1) * U * mag)).all()
    assert ex.smoe.smoe_last_device_status() == ex.smoe.SMOE_OK


@pytest.mark.parametrize("how", [{}, GROUPED, dict(norm=False)], ids=["softmax", "groups", "plain"])
@pytest.mark.parametrize("T", [1, 7, 64, 300])
def test_every_stage_of_the_layer(ex, T, how):
    gate, gate_up, down, bias, r = _weights(1)
    bias = bias if how else None
    layer = ex.F8Layer(gate, gate_up, down, K, 300, bias, **how)
    x = r(T, D)
    out = torch.full((T, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    layer(x, out)
    _stages(ex, layer, x, out, bias, how)


@pytest.mark.parametrize("n,d,d_ff,k", [(3, 80, 48, 1), (9, 144, 112, 3), (6, 272, 16, 6)])
@pytest.mark.parametrize("T", [1, 5, 70])
def test_odd_sizes(ex, T, n, d, d_ff, k):
    gate, gate_up, down, _, r = _weights(n, n, d, d_ff)
    layer = ex.F8Layer(gate, gate_up.to(torch.bfloat16), down, k, 70)
    x, out = r(T, d), torch.full((T, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    layer(x, out)
    _stages(ex, layer, x, out, None, {})


def test_experts_that_are_off_and_rows_without_an_order(ex):
    """Two experts of sixteen stay on: a token's other slots are empty and add
    nothing.  A token with a NaN has NaN outputs, and no other has."""
    gate, gate_up, down, bias, r = _weights(2)
    bias[:] = float("-inf")
    bias[3] = bias[9] = 0
    layer = ex.F8Layer(gate, gate_up, down, K, 40, bias)
    x, out = r(40, D), torch.full((40, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    layer(x, out)
    assert (layer.idx[:, 2:] == -1).all() and layer.offsets[-1] == 80
    _stages(ex, layer, x, out, bias, {})
    x[7, 5] = float("nan")
    other = torch.empty_like(out)
    layer(x, other)
    assert torch.isnan(other[7]).all()
    rest = torch.arange(40, device="cuda") != 7
    assert torch.equal(other[rest], out[rest])


@pytest.mark.parametrize("T", [3, 40, 300])
def test_the_layer_in_a_graph(ex, T):
    gate, gate_up, down, bias, r = _weights(3)
    layer = ex.F8Layer(gate, gate_up, down, K, T, bias, **GROUPED)
    x = r(T, D)
    out, eager = (torch.empty(T, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    layer(x, out, s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        layer(x, out, s)
    for _ in range(3):
        x.copy_(r(T, D))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        layer(x, eager)
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


def test_two_layers_at_once(ex):
    """On two streams, each with buffers of its own: the outputs of each alone."""
    gate, gate_up, down, bias, r = _weights(4)
    layers = [ex.F8Layer(gate, gate_up, down, K, 300, bias, **how) for how in ({}, GROUPED)]
    xs, streams = [r(300, D), r(300, D)], [torch.cuda.Stream() for _ in range(2)]
    alone = [layer(x, torch.empty(300, D, dtype=torch.bfloat16, device="cuda")) for layer, x in zip(layers, xs)]
    outs = [torch.empty(300, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for o in zip(layers, xs, outs, streams):
            o[0](*o[1:])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(alone, outs))


# ---------------------------------------------------------------- training

def _holds_as_a_gradient_of_weights(got, d_ys, xs, offsets):
    """The gradient of matrices against float64 of the rows that it was given."""
    at = offsets.tolist()
    for e in range(got.shape[0]):
        a, b = d_ys[at[e]:at[e + 1]].double(), xs[at[e]:at[e + 1]].double()
        ref, mag = a.t() @ b, a.abs().t() @ b.abs()
        err = (len(a) + 2) * 2.0 ** -23 * mag
        assert ((got[e].double() - ref).abs() <= err + ROUND[got.dtype] * (ref.abs() + err) + 1e-37).all()


def _product_stage(xs, w, offsets, ys, d_ys=None, d_xs=None, d_w=None):
    """A product and its gradients against float64 of the codes' values, quantised here."""
    n, n_out, n_in = w.shape
    w64 = torch.stack([_f64(_block_values(m)) for m in w.float().cpu().numpy()])
    rows = lambda t: _f64(u.rows_of(*u.quantize_rows(t.float().cpu().numpy())))  # noqa: E731
    assert _product_holds(ys, *_by_expert(rows(xs), w64, offsets), n_in)
    if d_xs is not None:
        assert _product_holds(d_xs, *_by_expert(rows(d_ys), w64.transpose(1, 2), offsets), n_out)
    if d_w is not None:
        _holds_as_a_gradient_of_weights(d_w, d_ys.to(torch.bfloat16), xs.to(torch.bfloat16), offsets)


def _block_values(w):
    """float64 values of a matrix after quantising its blocks of 128 x 128."""
    v = np.zeros(w.shape)
    for i in range(0, w.shape[0], 128):
        for j in range(0, w.shape[1], 128):
            q, s = u.quantize(w[i:i + 128, j:j + 128])
            v[i:i + 128, j:j + 128] = u.e4m3(q) * np.float64(s)
    return v


@pytest.mark.parametrize("x_type", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("w_type", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("counts,n_out,n_in", [([3, 0, 70, 1], 144, 80), ([0, 0], 16, 16), ([200], 272, 256)])
def test_the_product_and_its_gradients(ex, x_type, w_type, counts, n_out, n_in):
    g = torch.Generator(device="cuda").manual_seed(n_out)
    R = sum(counts) + 2  # two rows behind the last expert's
    xs = torch.randn(R, n_in, generator=g, device="cuda").to(x_type).requires_grad_()
    w = torch.randn(len(counts), n_out, n_in, generator=g, device="cuda").to(w_type).requires_grad_()
    offsets = torch.tensor([0, *np.cumsum(counts)], dtype=torch.int32, device="cuda")
    ys = ex.experts_f8(xs, w, offsets)
    d_ys = torch.randn(R, n_out, generator=g, device="cuda").to(x_type)
    ys.backward(d_ys)
    assert ys.dtype == xs.grad.dtype == x_type and w.grad.dtype == w_type
    _product_stage(xs.detach(), w.detach(), offsets, ys.detach(), d_ys, xs.grad, w.grad)
    assert not xs.grad[-2:].any() and not ys[-2:].any()
    for a, b in ((xs.detach(), w), (xs, w.detach())):  # one gradient alone
        one, = torch.autograd.grad(ex.experts_f8(a, b, offsets), b if b.requires_grad else a, d_ys)
        assert torch.equal(one, w.grad if b.requires_grad else xs.grad)
    assert ex.smoe.smoe_last_device_status() == ex.smoe.SMOE_OK


@pytest.mark.parametrize("score,norm", [(0, True), (0, False), (1, True), (1, False)])
def test_the_weights_of_the_routing_have_their_gradient(ex, score, norm):
    """Against differences of the float64 weights of the same choice."""
    T, n, k = 5, 12, 3
    g = torch.Generator(device="cuda").manual_seed(score)
    l = torch.randn(T, n, generator=g, device="cuda").requires_grad_()
    dw = torch.randn(T, k, generator=g, device="cuda")
    bias = torch.randn(n, generator=g, device="cuda")
    idx, w = ex.route(l, k, bias, score=score, n_groups=3, top_groups=2, group_best=2, norm=norm, scale=1.5)
    w.backward(dw)
    i, l64, d64 = idx.cpu().numpy(), l.detach().double().cpu().numpy(), dw.double().cpu().numpy()
    loss = lambda v: (u.weights(v, i, score == 0, norm, 1.5) * d64).sum()  # noqa: E731
    step = 2.0 ** -12
    for t in range(T):
        for e in range(n):
            p, m = l64.copy(), l64.copy()
            p[t, e] += step
            m[t, e] -= step
            # differences: a sixth of step^2 times a third derivative of at most 6 scale sum |dw|; f32: 2^-18 of the sum
            assert abs((loss(p) - loss(m)) / (2 * step) - l.grad[t, e].item()) <= (step ** 2 + 2.0 ** -18) * 1.5 * abs(d64[t]).sum()


def _train_inputs(x_type, T=61, n=8, d=144, d_ff=80):
    gate, gate_up, down, bias, r = _weights(5, n, d, d_ff)
    leaves = [r(T, d).to(x_type), gate.float(), gate_up, down]
    return [t.requires_grad_() for t in leaves], bias, r(T, d).to(x_type)


HOWS = [{}, dict(score=1, n_groups=4, top_groups=2, group_best=2, scale=2.5)]


@pytest.mark.parametrize("x_type", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("how", HOWS, ids=["softmax", "groups"])
def test_every_stage_of_a_training_step(ex, monkeypatch, x_type, how):
    """Each product, the routing and their gradients, against float64 of what came in."""
    leaves, bias, d_out = _train_inputs(x_type)
    x, router, gate_up, down = leaves
    seen, routed, product, rout = [], [], ex.experts_f8, ex.route

    def record(xs, w, offsets):
        if not xs.is_leaf:
            xs.retain_grad()
        ys = product(xs, w, offsets)
        ys.retain_grad()
        seen.append((xs, w, offsets, ys))
        return ys

    def record_route(logits, *a, **kw):
        logits.retain_grad()
        idx, w = rout(logits, *a, **kw)
        w.retain_grad()
        routed.append((logits, idx, w))
        return idx, w

    monkeypatch.setattr(ex, "experts_f8", record)
    monkeypatch.setattr(ex, "route", record_route)
    out = ex.moe_train_f8(*leaves, 3, bias, **how)
    out.backward(d_out)
    assert out.dtype == x.grad.dtype == x_type
    for xs, w, offsets, ys in seen:
        assert offsets[-1] == xs.shape[0]
        _product_stage(xs.detach(), w.detach(), offsets, ys.detach(), ys.grad, xs.grad, w.grad)
    (logits, idx, w), = routed
    soft, scale = how.get("score", 0) == 0, how.get("scale", 1.0)
    l, i = logits.detach().cpu().numpy(), idx.cpu().numpy()
    assert (i == u.choose(l, bias.cpu().numpy(), soft, how.get("n_groups", 1), how.get("top_groups", 1), how.get("group_best", 1),
                          3)).all()
    d, mag = u.weights_gradient(l, i, soft, True, scale, w.grad.double().cpu().numpy())
    assert (np.abs(logits.grad.cpu().numpy() - d) <= 4 * ((20 + 8 / 32 + 32) * 2 * U + 3 * 2.0 ** -23) * mag + 1e-36).all()
    assert ex.smoe.smoe_last_device_status() == ex.smoe.SMOE_OK


@pytest.mark.parametrize("how", HOWS, ids=["softmax", "groups"])
def test_a_training_step_in_a_graph(ex, how):
    """Forward and backward captured once, replayed on new inputs: the eager step's bits."""
    leaves, bias, d_out = _train_inputs(torch.bfloat16, T=300)
    step = lambda p: torch.autograd.grad(ex.moe_train_f8(*p, 3, bias, **how), p, d_out)  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(leaves)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        grads = step(leaves)
    for seed in range(3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        with torch.no_grad():
            leaves[0].copy_(torch.randn(leaves[0].shape, generator=g, device="cuda"))
            leaves[2].mul_(1.25)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        eager = step([p.detach().clone().requires_grad_() for p in leaves])
        assert all(torch.equal(a, b) for a, b in zip(grads, eager))
    assert ex.smoe.smoe_last_device_status() == ex.smoe.SMOE_OK


# ---------------------------------------------------------------- refusals

def test_a_capture_on_leaves_of_a_living_graph_is_refused(ex):
    """Torch's own additions to their gradients would end the process; refused before
    anything is captured, and not once that graph is gone."""
    leaves, bias, d_out = _train_inputs(torch.bfloat16)
    s = torch.cuda.Stream()
    living = ex.moe_train_f8(*leaves, 3, bias)
    torch.cuda.synchronize()
    with pytest.raises(RuntimeError, match="no eager graph holds"):
        with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=s):
            ex.moe_train_f8(*leaves, 3, bias)
    eager = torch.autograd.grad(living, leaves, d_out)
    del living
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        grads = torch.autograd.grad(ex.moe_train_f8(*leaves, 3, bias), leaves, d_out)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(grads, eager))
    with torch.no_grad():  # without gradients there is nothing to refuse
        out = ex.moe_train_f8(*leaves, 3, bias)
    assert not out.requires_grad and ex.smoe.smoe_last_device_status() == ex.smoe.SMOE_OK


def test_what_is_refused(ex):
    gate, gate_up, down, bias, r = _weights(6)
    for bad in ((gate.float(), gate_up, down), (gate[:-1], gate_up, down), (gate, gate_up[:, :-2], down),
                (gate, gate_up, down[:, :, :-16]), (gate, gate_up.half(), down), (gate, gate_up, down.cpu())):
        with pytest.raises((TypeError, ValueError)):
            ex.F8Layer(*bad, K, 8)
    for b in (bias.double(), bias[:-1], bias.cpu()):
        with pytest.raises((TypeError, ValueError)):
            ex.F8Layer(gate, gate_up, down, K, 8, b)
        with pytest.raises((TypeError, ValueError)):
            ex.route(r(4, N), K, b)
    layer, out = ex.F8Layer(gate, gate_up, down, K, 8), torch.full((9, D), -7.0, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="made for"):
        layer(r(9, D), out)
    for x, o in ((r(4, D).to(torch.bfloat16), out[:4]), (r(4, 2 * D)[:, :D], out[:4]), (r(4, D), out[:3]), (r(4, D).cpu(), out[:4])):
        with pytest.raises((TypeError, ValueError)):
            layer(x, o)
    offsets = torch.zeros(N + 1, dtype=torch.int32, device="cuda")
    for xs, w, o in ((r(4, D).half(), gate_up, offsets), (r(4, D), gate_up[..., :-16], offsets), (r(4, D), gate_up, offsets.long()),
                     (r(4, D), gate_up, offsets[1:]), (r(4, 24), r(N, 32, 24), offsets), (r(4, 32), r(N, 24, 32), offsets)):
        with pytest.raises((TypeError, ValueError)):
            ex.experts_f8(xs, w, o)
    for how in (dict(score=2), dict(n_groups=3), dict(n_groups=4, top_groups=5), dict(group_best=3), dict(scale=0.0)):
        with pytest.raises(ex.smoe.SmoeError):
            ex.route(r(4, N), K, **how)
    torch.cuda.synchronize()
    assert (out == -7).all()
    assert layer(r(0, D), out[:0]).shape == (0, D)
    assert ex.smoe.smoe_last_device_status() == ex.smoe.SMOE_OK


@pytest.mark.parametrize("which", ["route", "experts_f8"])
def test_a_second_gradient_is_refused(ex, which):
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").requires_grad_()  # noqa: E731
    l, xs, w = r(6, 8), r(12, 16), r(2, 16, 16)
    offsets = torch.tensor([0, 5, 12], dtype=torch.int32, device="cuda")
    out, arg = (ex.route(l, 2)[1], l) if which == "route" else (ex.experts_f8(xs, w, offsets), w)
    first, = torch.autograd.grad(out.square().sum(), arg, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        first.square().sum().backward()
