"""Parity of the many-token calls with plain float64 forms, through the C ABI.

Tolerances, from the arithmetic (u = 2^-24, f32 rounding; a bf16 output adds
2^-8 of its value):
* top_w: the exponent's subtraction is off by u |l - l0|, exp by 2 units in
  the last place, the sum of k by 7 roundings (two per lane, five shuffles),
  the division by one: u (max |l - l0| + 16) relative.
* sums over k slots: k + 1 roundings of sum |w y|.
* dots over d: at most d / 32 + 7 roundings of sum |g y| (32 lanes in chains).
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f32": (0, torch.float32, 0.0), "bf16": (1, torch.bfloat16, 2.0 ** -8)}


@pytest.fixture(scope="module")
def smoe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build_library()
    import moe_expert_ffn_smoe_gb300 as m
    return m


@pytest.fixture(autouse=True)
def _no_device_error(smoe):
    yield
    assert smoe.smoe_last_device_status() == smoe.SMOE_OK


def _guarded(shape, dtype, fill):
    """A tensor of `shape` with 64 guard elements after it."""
    n = int(np.prod(shape))
    buf = torch.full((n + 64,), fill, dtype=dtype, device="cuda")
    return buf[:n].view(*shape), buf[n:]


def _intact(guard, fill):
    g = guard.float()
    assert (torch.isnan(g) if np.isnan(fill) else g == fill).all(), "written past the end"


# ---------------------------------------------------------------- selection

def _select_ref(l, k):
    T, E = l.shape
    nan = np.isnan(l)
    key = np.where(nan, -np.inf, l)
    take = np.lexsort((np.broadcast_to(np.arange(E), l.shape), -key, nan), axis=1)[:, :k]
    v = np.take_along_axis(l, take, 1).astype(np.float64)
    there = v != -np.inf
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.where(there, np.exp(v - np.where(there[:, :1], v[:, :1], 0.0)), 0.0)
        s = w.sum(1, keepdims=True)
        w = np.where(s == 0, 0.0, w / np.where(s == 0, 1.0, s))
    return np.where(there, take, -1), w


def _logits(T, E, seed, masked=False, ties=False):
    rng = np.random.default_rng([seed, T, E])
    l = rng.normal(size=(T, E)).astype(np.float32)
    if ties:
        l = np.round(l * 2) / 2
    if masked:
        l[rng.random((T, E)) < 0.3] = -np.inf
        l[rng.random(T) < 0.2] = -np.inf
    return l


def _topk(smoe, l, k, ld=None):
    T, E = l.shape
    ld = ld or E
    src = torch.full((T, ld), float("inf"), device="cuda")
    src[:, :E] = torch.from_numpy(l).cuda()
    idx, gi = _guarded((T, k), torch.int32, -7)
    w, gw = _guarded((T, k), torch.float32, float("nan"))
    smoe.smoe_topk_rows(src, T, E, ld, k, idx, w)
    torch.cuda.synchronize()
    _intact(gi, -7)
    _intact(gw, float("nan"))
    return idx, w


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 128, 8), (7, 128, 8), (33, 64, 6), (9, 65, 1), (5, 256, 64), (130, 129, 33),
                                   (17, 512, 16), (6, 513, 9), (3, 8192, 64), (2000, 128, 8), (4, 40, 40)])
@pytest.mark.parametrize("kind", ["plain", "masked", "ties"])
def test_topk_rows(smoe, T, E, k, kind):
    l = _logits(T, E, 1, masked=kind == "masked", ties=kind == "ties")
    idx, w = _topk(smoe, l, k, ld=E + (5 if kind == "ties" else 0))
    ri, rw = _select_ref(l, k)
    np.testing.assert_array_equal(idx.cpu().numpy(), ri)
    span = np.nanmax(np.where(np.isfinite(l), l, np.nan)) - np.nanmin(np.where(np.isfinite(l), l, np.nan)) if np.isfinite(l).any() else 0
    np.testing.assert_allclose(w.cpu().numpy(), rw, rtol=U * (span + 16), atol=1e-37)


@pytest.mark.parametrize("T,E,k", [(9, 513, 16), (70, 8192, 8), (5, 2047, 16), (1030, 2048, 3), (5, 2049, 16), (33, 1000, 17),
                                   (4, 5000, 40)])
@pytest.mark.parametrize("kind", ["plain", "masked", "ties"])
def test_topk_of_many_experts(smoe, T, E, k, kind):
    l = _logits(T, E, 22, masked=kind == "masked", ties=kind == "ties")
    idx, w = _topk(smoe, l, k, ld=E + 3)
    ri, rw = _select_ref(l, k)
    np.testing.assert_array_equal(idx.cpu().numpy(), ri)
    np.testing.assert_allclose(w.cpu().numpy(), rw, rtol=U * (12 + 16), atol=1e-37)  # |l| < 6


@pytest.mark.parametrize("T,E,k", [(10001, 128, 8), (12003, 64, 3), (10002, 40, 16), (9999, 256, 9), (10003, 512, 1), (9730, 128, 8)])
@pytest.mark.parametrize("kind", ["plain", "masked", "ties"])
def test_topk_of_many_rows(smoe, T, E, k, kind):
    """More rows than a wave of warps."""
    l = _logits(T, E, 21, masked=kind == "masked", ties=kind == "ties")
    idx, w = _topk(smoe, l, k)
    ri, rw = _select_ref(l, k)
    np.testing.assert_array_equal(idx.cpu().numpy(), ri)
    np.testing.assert_allclose(w.cpu().numpy(), rw, rtol=U * (12 + 16), atol=1e-37)  # |l| < 6


@pytest.mark.parametrize("E", [20, 600])
def test_topk_rows_nan_and_infinities(smoe, E):
    l = np.full((4, E), -np.inf, np.float32)
    l[0, 3] = 1.0                      # one expert left of k
    l[1, 5], l[1, 2] = np.nan, -2.0    # NaN ranks below every number, -inf among them
    l[2, :] = np.nan
    l[3, :] = np.float32(-3.4028235e38)  # the type's lowest value is a number
    idx, w = _topk(smoe, l, 3)
    i, w = idx.cpu().numpy(), w.cpu().numpy()
    assert i[0].tolist() == [3, -1, -1] and w[0].tolist() == [1, 0, 0]
    assert i[1].tolist() == [2, -1, -1] and w[1].tolist() == [1, 0, 0]
    assert i[2].tolist() == [0, 1, 2] and np.isnan(w[2]).all()
    assert i[3].tolist() == [0, 1, 2]
    np.testing.assert_allclose(w[3], 1 / 3, rtol=U * 16)


@pytest.mark.parametrize("T,E,k,masked", [(1, 1, 1, False), (5, 128, 8, True), (37, 33, 5, True), (200, 512, 16, False),
                                          (3, 700, 40, True), (9, 6, 6, False)])
def test_topk_rows_gradient(smoe, T, E, k, masked):
    l = _logits(T, E, 2, masked=masked)
    idx, w = _topk(smoe, l, k)
    rng = np.random.default_rng(3)
    dw = rng.normal(size=(T, k)).astype(np.float32)
    dl, g = _guarded((T, E), torch.float32, float("nan"))
    smoe.smoe_topk_rows_backward(idx, w, torch.from_numpy(dw).cuda(), T, E, k, dl)
    got = dl.cpu().numpy().astype(np.float64)
    _intact(g, float("nan"))
    ri, rw = _select_ref(l, k)
    ref = np.zeros((T, E))
    mag = np.zeros((T, E))
    for t in range(T):
        c = (rw[t] * dw[t]).sum()
        for r in range(k):
            if ri[t, r] >= 0:
                ref[t, ri[t, r]] = rw[t, r] * (dw[t, r] - c)
                mag[t, ri[t, r]] = rw[t, r] * (abs(dw[t, r]) + (rw[t] * np.abs(dw[t])).sum())
    # w itself is off by u (span + 16) with span < 16 here, twice (in c and as the factor), and 8 roundings
    assert (np.abs(got - ref) <= U * 72 * mag + 1e-37).all()
    assert (got[ref == 0] == 0).all()
    # and against differences of the float64 weights, the selection held
    h = 1e-5
    for t in range(min(T, 4)):
        for r in range(min(k, 6)):
            if ri[t, r] < 0:
                continue
            f = []
            for sgn in (1, -1):
                v = l[t].astype(np.float64)
                v[ri[t, r]] += sgn * h
                sel = ri[t][ri[t] >= 0]
                e = np.exp(v[sel] - v[sel].max())
                f.append(((e / e.sum()) * dw[t][ri[t] >= 0]).sum())
            # the difference: h^2 of a third derivative below 6 max|dw|, and 2^-52 / h of rounding
            tol = 6 * h * h * np.abs(dw[t]).max() + 1e-9 + U * 72 * mag[t, ri[t, r]]
            assert abs((f[0] - f[1]) / (2 * h) - got[t, ri[t, r]]) <= tol


# ---------------------------------------------------------------- dispatch

def _indices(T, k, E, seed, kind):
    rng = np.random.default_rng([seed, T, k, E])
    idx = np.stack([rng.permutation(max(E, k))[:k] % E for _ in range(T)]).astype(np.int32).reshape(T, k)
    if kind == "dropped":
        idx[rng.random((T, k)) < 0.2] = -1
        idx[rng.random(T) < 0.2] = -1
        idx[rng.random((T, k)) < 0.02] = E + 3
    elif kind == "one":
        idx[:] = E - 1
    elif kind == "none":
        idx[:] = -1
    return idx


def _sort_ref(idx, E):
    a = idx.reshape(-1)
    key = np.where((a >= 0) & (a < E), a, E)
    order = np.argsort(key, kind="stable")
    at = np.empty(a.size, np.int64)
    at[order] = np.arange(a.size)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=E + 1)[:E])])
    return offsets, order, np.where(key < E, at, -1 - at)


def _dispatch(smoe, idx, E, x=None, dt="f32"):
    T, k = idx.shape
    d = x.shape[1] if x is not None else 0
    offsets, g0 = _guarded((E + 1,), torch.int32, -7)
    order, g1 = _guarded((T * k,), torch.int32, -7)
    place, g2 = _guarded((T, k), torch.int32, -7)
    xs, g3 = _guarded((T * k, d), DT[dt][1], -7.0)
    need = smoe.smoe_dispatch_workspace_bytes(T, k, E)
    ws, g4 = _guarded((need,), torch.uint8, 201)
    smoe.smoe_dispatch_tokens(torch.from_numpy(idx).cuda(), T, k, E, x, DT[dt][0], d, offsets, order, place,
                              xs if x is not None else None, ws, need)
    torch.cuda.synchronize()
    for g in (g0, g1, g2, g3):
        _intact(g, -7)
    _intact(g4, 201)
    return offsets, order, place, xs


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 128), (16, 8, 128), (33, 2, 5), (300, 8, 128), (1000, 3, 7), (129, 64, 64),
                                   (2049, 6, 200), (40, 4, 8192), (9000, 8, 300), (31, 8, 33), (32, 8, 33)])
@pytest.mark.parametrize("kind", ["all", "dropped", "one", "none"])
def test_sort(smoe, T, k, E, kind):
    idx = _indices(T, k, E, 4, kind)
    offsets, order, place, _ = _dispatch(smoe, idx, E)
    ro, rr, rp = _sort_ref(idx, E)
    np.testing.assert_array_equal(offsets.cpu().numpy(), ro)
    np.testing.assert_array_equal(order.cpu().numpy(), rr)
    np.testing.assert_array_equal(place.cpu().numpy().reshape(-1), rp)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,k,E,d", [(1, 1, 1, 1), (5, 8, 128, 4096), (37, 3, 6, 100), (64, 8, 32, 513), (3, 2, 4, 9000),
                                     (700, 8, 128, 64), (16, 64, 128, 24)])
@pytest.mark.parametrize("kind", ["all", "dropped", "none"])
def test_dispatch_rows_and_gradient(smoe, dt, T, k, E, d, kind):
    idx = _indices(T, k, E, 5, kind)
    _, tt, eps = DT[dt]
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(T, d, generator=g, device="cuda").to(tt)
    x[0, 0] = float("inf")
    x[-1, -1] = float("nan")
    offsets, order, place, xs = _dispatch(smoe, idx, E, x, dt)
    there = place.reshape(-1)[order.long()] >= 0
    ref = torch.where(there[:, None], x[order.long() // k], torch.zeros((), dtype=tt, device="cuda"))
    assert torch.equal(xs.nan_to_num(7.5), ref.nan_to_num(7.5))

    d_xs = torch.randn(T * k, d, generator=g, device="cuda").to(tt)
    d_xs[~there] = float("nan")  # rows without an expert are not read
    d_x, guard = _guarded((T, d), tt, -7.0)
    smoe.smoe_dispatch_tokens_backward(d_xs, DT[dt][0], place, T, k, d, d_x)
    torch.cuda.synchronize()
    _intact(guard, -7)
    p = place.long()
    rows = torch.where((p >= 0)[..., None], d_xs[p.clamp(min=0)].double(), 0.0)
    ref, mag = rows.sum(1), rows.abs().sum(1)
    assert ((d_x.double() - ref).abs() <= U * (k + 1) * mag + eps * ref.abs()).all()


def test_dispatch_of_no_tokens_writes_zero_offsets(smoe):
    offsets = torch.full((129,), -7, dtype=torch.int32, device="cuda")
    smoe.smoe_dispatch_tokens(None, 0, 8, 128, None, 0, 64, offsets, None, None, None, None, 0)
    assert (offsets == 0).all()


# ---------------------------------------------------------------- combine

@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,k,E,d", [(1, 1, 1, 1), (16, 8, 128, 4096), (37, 3, 6, 100), (64, 8, 32, 513), (3, 2, 4, 9000),
                                     (300, 8, 128, 64), (16, 64, 128, 24), (2, 9, 16, 2056)])
@pytest.mark.parametrize("kind", ["all", "dropped", "none"])
def test_combine_and_gradients(smoe, dt, T, k, E, d, kind):
    code, tt, eps = DT[dt]
    idx = _indices(T, k, E, 7, kind)
    _, order, place, _ = _dispatch(smoe, idx, E)
    p = place.long()
    there = p >= 0
    g = torch.Generator(device="cuda").manual_seed(8)
    w = torch.rand(T, k, generator=g, device="cuda")
    w[~there] = float("nan")  # not read where the slot has no expert
    ys = torch.randn(T * k, d, generator=g, device="cuda").to(tt)
    ys[~there.reshape(-1)[order.long()]] = float("nan")
    out, go = _guarded((T, d), tt, -7.0)
    smoe.smoe_combine_tokens(ys, code, place, w, T, k, d, out)
    torch.cuda.synchronize()
    _intact(go, -7)
    rows = torch.where(there[..., None], ys[p.clamp(min=0)].double(), 0.0)
    wd = torch.where(there, w.double(), 0.0)
    prod = rows * wd[..., None]
    ref = prod.sum(1)
    assert ((out.double() - ref).abs() <= U * (k + 1) * prod.abs().sum(1) + eps * ref.abs()).all()

    d_out = torch.randn(T, d, generator=g, device="cuda").to(tt)
    d_ys, g1 = _guarded((T * k, d), tt, -7.0)
    d_w, g2 = _guarded((T, k), torch.float32, -7.0)
    smoe.smoe_combine_tokens_backward(d_out, ys, code, place, w, T, k, d, d_ys, d_w)
    torch.cuda.synchronize()
    _intact(g1, -7)
    _intact(g2, -7)
    ref_y = torch.zeros(T * k, d, dtype=torch.float64, device="cuda")
    ref_y[p[there]] = (d_out.double()[:, None, :] * wd[..., None])[there]
    assert ((d_ys.double() - ref_y).abs() <= (U + eps) * ref_y.abs()).all()
    dots = d_out.double()[:, None, :] * rows
    assert ((d_w.double() - dots.sum(2)).abs() <= U * (d / 32 + 7) * dots.abs().sum(2)).all()
    assert (d_w[~there] == 0).all()


def test_combine_gradient_against_differences(smoe):
    """The combine is linear in ys and in w: its own differences along a
    direction are the gradient's product with it, up to f32 rounding."""
    T, k, E, d = 9, 4, 6, 80
    idx = _indices(T, k, E, 9, "dropped")
    _, _, place, _ = _dispatch(smoe, idx, E)
    g = torch.Generator(device="cuda").manual_seed(10)
    ys, dy = (torch.randn(T * k, d, generator=g, device="cuda") for _ in range(2))
    w, dw = (torch.randn(T, k, generator=g, device="cuda") for _ in range(2))
    d_out = torch.randn(T, d, generator=g, device="cuda")

    def f(a, b):
        out = torch.empty(T, d, device="cuda")
        smoe.smoe_combine_tokens(a, 0, place, b, T, k, d, out)
        return (out.double() * d_out.double()).sum().item()

    gy, gw = torch.empty_like(ys), torch.empty_like(w)
    smoe.smoe_combine_tokens_backward(d_out, ys, 0, place, w, T, k, d, gy, gw)
    # each forward is off by at most u (k + 1) sum |d_out w y|, inputs y +- dy by u |.|
    mag = (d_out.abs().double().sum() * 4 * 4 * k).item()  # |w|, |y| <= 4 + 4 on 99.99% and far less on average
    tol = U * (k + 3) * mag
    assert abs((f(ys + dy, w) - f(ys - dy, w)) / 2 - (gy.double() * dy.double()).sum().item()) <= tol
    assert abs((f(ys, w + dw) - f(ys, w - dw)) / 2 - (gw.double() * dw.double()).sum().item()) <= tol


def test_places_out_of_range_are_reported_not_followed(smoe):
    T, k, d = 4, 2, 32
    place = torch.tensor([[0, 1], [2, 99], [-50, 3], [-1, 5]], dtype=torch.int32, device="cuda")
    ys = torch.ones(T * k, d, device="cuda")
    w = torch.ones(T, k, device="cuda")
    out = torch.empty(T, d, device="cuda")
    smoe.smoe_combine_tokens(ys, 0, place, w, T, k, d, out)
    assert smoe.smoe_last_device_status() == smoe.SMOE_ERR_ROUTE
    assert out[:, 0].tolist() == [2, 1, 1, 1]
    d_ys, d_w = torch.empty(T * k, d, device="cuda"), torch.empty(T, k, device="cuda")
    smoe.smoe_combine_tokens_backward(out, ys, 0, place, w, T, k, d, d_ys, d_w)
    assert smoe.smoe_last_device_status() == smoe.SMOE_ERR_ROUTE
    assert d_w.tolist() == [[64, 64], [32, 0], [0, 32], [0, 32]]


def test_side_stream_and_graph(smoe):
    """The whole chain on a stream of its own, captured and replayed on new logits."""
    T, E, k, d = 50, 32, 4, 96
    s = torch.cuda.Stream()
    g = torch.Generator(device="cuda").manual_seed(11)
    l = torch.randn(T, E, generator=g, device="cuda")
    x = torch.randn(T, d, generator=g, device="cuda")
    idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w, out = torch.empty(T, k, device="cuda"), torch.empty(T, d, device="cuda")
    offsets = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    order, place = (torch.empty(T * k, dtype=torch.int32, device="cuda") for _ in range(2))
    xs = torch.empty(T * k, d, device="cuda")
    need = smoe.smoe_dispatch_workspace_bytes(T, k, E)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def chain():
        smoe.smoe_topk_rows(l, T, E, E, k, idx, w, stream=s)
        smoe.smoe_dispatch_tokens(idx, T, k, E, x, 0, d, offsets, order, place, xs, ws, need, stream=s)
        smoe.smoe_combine_tokens(xs, 0, place, w, T, k, d, out, stream=s)

    torch.cuda.synchronize()
    chain()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        chain()
    for _ in range(3):
        l.copy_(torch.randn(T, E, generator=g, device="cuda"))
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        # weights that sum to one on copies of the row give the row back
        ref = x.double()
        assert ((out.double() - ref).abs() <= U * 32 * ref.abs()).all()


@pytest.mark.parametrize("T,k,E", [(3000, 4, 8192), (1024, 4, 64), (1025, 4, 64), (70000, 2, 33)])
def test_sort_of_many(smoe, T, k, E):
    """Many buckets, many chunks."""
    for kind in ("all", "dropped"):
        idx = _indices(T, k, min(E, 64), 12, kind) if E <= 64 else _indices(T, k, E, 12, kind)
        offsets, order, place, _ = _dispatch(smoe, idx, E)
        ro, rr, rp = _sort_ref(idx, E)
        np.testing.assert_array_equal(offsets.cpu().numpy(), ro)
        np.testing.assert_array_equal(order.cpu().numpy(), rr)
        np.testing.assert_array_equal(place.cpu().numpy().reshape(-1), rp)


@pytest.mark.parametrize("T,k,E", [(192, 8, 64), (193, 8, 64), (4096, 8, 128), (4097, 8, 128), (16384, 8, 128), (16385, 8, 128), (10000, 4, 8192),
                                   (33000, 4, 8192), (520, 63, 64),
                                   (33000, 1, 5)])
@pytest.mark.parametrize("kind", ["all", "dropped", "one", "none"])
def test_sort_at_the_forms_borders(smoe, T, k, E, kind):
    """The first and last sizes of the two-launch dispatch (1537 to 32,768
    slots) and those around them, with rows of their own so that both the sort and the copy are seen."""
    idx = _indices(T, k, E, 14, kind)
    x = torch.arange(T, device="cuda", dtype=torch.float32)[:, None].expand(T, 4).contiguous()
    offsets, order, place, xs = _dispatch(smoe, idx, E, x)
    ro, rr, rp = _sort_ref(idx, E)
    np.testing.assert_array_equal(offsets.cpu().numpy(), ro)
    np.testing.assert_array_equal(order.cpu().numpy(), rr)
    np.testing.assert_array_equal(place.cpu().numpy().reshape(-1), rp)
    there = rp[rr] >= 0
    np.testing.assert_array_equal(xs[:, 3].cpu().numpy(), np.where(there, rr // k, 0))


def test_rows_past_32_bits(smoe):
    """5.3 GB of sorted rows: out and back."""
    T, k, E, d = 8200, 8, 16, 40000
    idx = _indices(T, k, E, 13, "all")
    g = torch.Generator(device="cuda").manual_seed(13)
    x = torch.randn(T, d, generator=g, device="cuda").to(torch.bfloat16)
    offsets, order, place, xs = _dispatch(smoe, idx, E, x, "bf16")
    for at in (0, T * k // 2, T * k - 64):
        assert torch.equal(xs[at:at + 64], x[order[at:at + 64].long() // k])
    w = torch.full((T, k), 1 / k, device="cuda")
    out = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    smoe.smoe_combine_tokens(xs, 1, place, w, T, k, d, out)
    assert torch.equal(out, x)  # eight eighths of a bf16 are exact
    d_ys, d_w = torch.empty_like(xs), torch.empty(T, k, device="cuda")
    smoe.smoe_combine_tokens_backward(x, xs, 1, place, w, T, k, d, d_ys, d_w)
    torch.cuda.synchronize()
    at = T * k - 64
    assert torch.equal(d_ys[at:], (x[order[at:].long() // k].float() / k).to(torch.bfloat16))
    ref = (x.double() ** 2).sum(1)
    assert ((d_w.double() - ref[:, None]).abs() <= U * (d / 32 + 7) * ref[:, None]).all()
