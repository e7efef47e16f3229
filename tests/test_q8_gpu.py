"""Parity of the 8-bit calls with plain float64 forms, through the C ABI.

The quantised codes are integers defined by f32 arithmetic (127 / top and its
product with v, each rounded once), so they are compared bit for bit.  The
products' sums are exact while they stay below 2^24; above, an f32 sum of K
terms is off by at most (K / 16) u of sum |xq wq| (u = 2^-24, one rounding
per step of 16 columns) plus 16 u of the largest; two scale factors and the
store add 3 u (2^-8 for bf16).
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


def _quantize(smoe, x, dt, act, cols):
    rows = x.shape[0]
    buf = torch.full((rows * cols + 64,), 99, dtype=torch.int8, device="cuda")
    s = torch.full((rows + 16,), -7.0, device="cuda")
    smoe.smoe_quantize_rows_q8(x, DT[dt][0], act, rows, cols, buf, s)
    torch.cuda.synchronize()
    assert (buf[rows * cols:] == 99).all() and (s[rows:] == -7).all()
    return buf[:rows * cols].view(rows, cols).cpu().numpy(), s[:rows].cpu().numpy()


def _quantize_ref(v):
    top = np.abs(v).max(1, keepdims=True, initial=0).astype(np.float32)
    up = np.where(top > 0, np.float32(127) / np.where(top > 0, top, 1), np.float32(0)).astype(np.float32)
    return np.rint((v * up).astype(np.float32)).astype(np.int8), (top / np.float32(127))[:, 0]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 4096), (7, 100), (33, 513), (3, 9000), (2, 32768), (300, 64)])
def test_quantize_rows(smoe, dt, rows, cols):
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, cols, generator=g, device="cuda").to(DT[dt][1])
    if rows > 2:
        x[1] = 0
        x[2, 0] = x[2].abs().max() * 2  # others at ties of the grid
    q, s = _quantize(smoe, x, dt, smoe.SMOE_Q8_PLAIN, cols)
    rq, rs = _quantize_ref(x.float().cpu().numpy())
    np.testing.assert_array_equal(q, rq)
    np.testing.assert_array_equal(s, rs)


def test_quantize_rows_that_are_not_finite(smoe):
    x = torch.ones(4, 96, device="cuda")
    x[0, 95] = float("nan")
    x[1, 3] = float("inf")
    x[2, 50] = 3.4e38
    q, s = _quantize(smoe, x, "f32", smoe.SMOE_Q8_PLAIN, 96)
    assert np.isnan(s[:2]).all() and (q[:2] == 0).all()
    assert np.isfinite(s[2:]).all() and q[2, 50] == 127 and (q[3] == 127).all()
    tiny = torch.full((1, 32), 1e-44, device="cuda")  # 127 / top overflows: the codes saturate
    q, s = _quantize(smoe, tiny, "f32", smoe.SMOE_Q8_PLAIN, 32)
    assert (q == 127).all() and s[0] >= 0


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 16), (5, 1536), (9, 101)])
def test_quantize_silu_mul(smoe, dt, rows, cols):
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, 2 * cols, generator=g, device="cuda").to(DT[dt][1])
    q, s = _quantize(smoe, x, dt, smoe.SMOE_Q8_SILU_MUL, cols)
    v = x.double().cpu().numpy()
    ga, up = v[:, :cols], v[:, cols:]
    ref = ga / (1 + np.exp(-ga)) * up
    top = np.abs(ref).max(1)
    # exp, the sum, the division and the product: 8 roundings at most
    np.testing.assert_allclose(s, top / 127, rtol=10 * U)
    # half a step, and the roundings of a value of up to 127 steps
    assert (np.abs(q * (top / 127)[:, None] - ref) <= (0.5 + 127 * 20 * U) * (top / 127)[:, None]).all()


def _codes(rows, cols, seed, full=False):
    rng = np.random.default_rng([seed, rows, cols])
    if full:
        return np.full((rows, cols), -128 if full == "low" else 127, np.int8)
    return np.clip(np.rint(rng.normal(size=(rows, cols)) * 40), -128, 127).astype(np.int8)


def _check(y, dt, ref, mag, K):
    eps = DT[dt][2]
    exact = 3 * U * np.abs(ref) + eps * np.abs(ref)
    big = np.where(mag[1] >= 2 ** 24, (K / 16 + 16) * U, 0.0) * mag[0]
    err = np.abs(y.double().cpu().numpy() - ref)
    assert (err <= exact + big).all(), float(np.max(err / (exact + big + 1e-30)))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("R,N,K", [(1, 1, 16), (1, 8192, 4096), (2, 129, 48), (8, 100, 4096), (9, 257, 1040), (16, 128, 64),
                                   (31, 1000, 528), (64, 512, 512), (100, 96, 2064), (129, 130, 144), (257, 384, 4096),
                                   (300, 77, 32), (3, 40, 32768), (70, 200, 32768), (512, 640, 112)])
def test_matmul(smoe, dt, R, N, K):
    x, w = _codes(R, K, 1), _codes(N, K, 2)
    rng = np.random.default_rng(3)
    xs, ws = rng.uniform(0.5, 2, R).astype(np.float32), rng.uniform(0.5, 2, N).astype(np.float32)
    y = torch.full((R * N + 64,), -7.0, dtype=DT[dt][1], device="cuda")
    need = smoe.smoe_matmul_q8_workspace_bytes(R, N, K)
    wsp = torch.full((need + 64,), 201, dtype=torch.uint8, device="cuda")
    c = lambda a: torch.from_numpy(a).cuda()
    smoe.smoe_matmul_q8(c(x), c(xs), R, c(w), c(ws), N, K, y, DT[dt][0], wsp, need)
    torch.cuda.synchronize()
    assert (y[R * N:] == -7).all() and (wsp[need:] == 201).all()
    s = np.outer(xs.astype(np.float64), ws)
    dot = x.astype(np.float64) @ w.astype(np.float64).T
    mag = np.abs(x.astype(np.float64)) @ np.abs(w.astype(np.float64)).T
    _check(y[:R * N].view(R, N), dt, dot * s, (mag * s, mag), K)


@pytest.mark.parametrize("R", [3, 40, 200])
def test_matmul_at_the_ends_of_the_codes(smoe, R):
    """Every product at its largest: 128 * 128 and -128 * 127 over 4096 columns."""
    N, K = 130, 4096
    one = torch.ones(512, device="cuda")
    for a, b in (("low", "low"), ("low", "high")):
        x, w = _codes(R, K, 0, full=a), _codes(N, K, 0, full=b)
        y = torch.empty(R, N, device="cuda")
        need = smoe.smoe_matmul_q8_workspace_bytes(R, N, K)
        wsp = torch.empty(need, dtype=torch.uint8, device="cuda")
        smoe.smoe_matmul_q8(torch.from_numpy(x).cuda(), one, R, torch.from_numpy(w).cuda(), one, N, K, y, 0, wsp, need)
        ref = float(int(x[0, 0]) * int(w[0, 0]) * K)
        assert ((y.double() - ref).abs() <= (K / 16 + 16) * U * abs(ref)).all()


def test_matmul_of_no_columns_and_of_rows_that_are_not_finite(smoe):
    one = torch.ones(64, device="cuda")
    y = torch.full((3, 40), 5.0, device="cuda")
    need = smoe.smoe_matmul_q8_workspace_bytes(3, 40, 0)
    wsp = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    smoe.smoe_matmul_q8(None, one, 3, None, one, 40, 0, y, 0, wsp, need)
    assert (y == 0).all()
    for R in (3, 40):
        s = torch.ones(R, device="cuda")
        s[1] = float("nan")
        x = torch.zeros(R, 64, dtype=torch.int8, device="cuda")
        w = torch.ones(40, 64, dtype=torch.int8, device="cuda")
        y = torch.empty(R, 40, device="cuda")
        need = smoe.smoe_matmul_q8_workspace_bytes(R, 40, 64)
        wsp = torch.empty(need, dtype=torch.uint8, device="cuda")
        smoe.smoe_matmul_q8(x, s, R, w, one, 40, 64, y, 0, wsp, need)
        assert torch.isnan(y[1]).all() and (y[0] == 0).all() and (y[2:] == 0).all()


def _experts(smoe, counts, tail, N, K, dt, k=0, seed=5, nsrc=None):
    """Rows of experts by `counts` and `tail` rows of none; k > 0: gathered."""
    E = len(counts)
    R = int(sum(counts)) + tail
    rng = np.random.default_rng([seed, R, N, K])
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    if k:
        T = -(-R // k)
        order = rng.permutation(T * k)[:R].astype(np.int32)
        src = order // k
    else:
        T, order, src = R, None, np.arange(R)
    x, w = _codes(T, K, seed), _codes(E * N, K, seed + 1)
    xs, ws = rng.uniform(0.5, 2, T).astype(np.float32), rng.uniform(0.5, 2, E * N).astype(np.float32)
    c = lambda a: torch.from_numpy(a).cuda()
    y = torch.full((R * N + 64,), -7.0, dtype=DT[dt][1], device="cuda")
    need = smoe.smoe_experts_matmul_q8_workspace_bytes(T, R, E, N, K)
    wsp = torch.full((need + 64,), 201, dtype=torch.uint8, device="cuda")
    smoe.smoe_experts_matmul_q8(c(x), c(xs), T, c(order) if k else None, max(k, 1), c(offsets), R, E, c(w), c(ws), N, K, y,
                                DT[dt][0], wsp, need)
    torch.cuda.synchronize()
    assert (y[R * N:] == -7).all() and (wsp[need:] == 201).all()
    y = y[:R * N].view(R, N)
    assert (y[offsets[-1]:] == 0).all()
    for e in range(E):
        a, b = offsets[e], offsets[e + 1]
        if a == b:
            continue
        xe, we = x[src[a:b]].astype(np.float64), w[e * N:(e + 1) * N].astype(np.float64)
        s = np.outer(xs[src[a:b]].astype(np.float64), ws[e * N:(e + 1) * N])
        mag = np.abs(xe) @ np.abs(we).T
        _check(y[a:b], dt, (xe @ we.T) * s, (mag * s, mag), K)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("k", [0, 1, 8])
@pytest.mark.parametrize("counts,tail,N,K", [
    ([1], 0, 16, 16),
    ([0, 0, 3, 0], 2, 129, 528),            # empty experts before and after
    ([0, 0], 5, 40, 64),                    # no row has an expert
    ([1, 0, 2, 8, 9, 0, 17], 3, 200, 1040),
    ([5] * 40, 0, 96, 256),
    ([130, 1, 0, 64, 257], 7, 300, 400),
    ([0, 300, 0], 1, 128, 4096),
    ([33] * 9, 0, 513, 272),
    ([1, 1] * 600, 4, 24, 32),              # more experts than one pass of the plan takes
    ([900, 2, 3], 0, 130, 128),
])
def test_experts_matmul(smoe, dt, k, counts, tail, N, K):
    _experts(smoe, counts, tail, N, K, dt, k)


def test_experts_matmul_reports_bad_orders_and_offsets(smoe):
    N, K, R, E = 64, 64, 40, 3
    one = torch.ones(E * N, device="cuda")
    x = torch.ones(R, K, dtype=torch.int8, device="cuda")
    w = torch.ones(E * N, K, dtype=torch.int8, device="cuda")
    need = smoe.smoe_experts_matmul_q8_workspace_bytes(R, R, E, N, K)
    wsp = torch.empty(need, dtype=torch.uint8, device="cuda")
    y = torch.empty(R, N, device="cuda")
    order = torch.arange(R, dtype=torch.int32, device="cuda")
    order[3], order[20] = 1000, -4
    off = torch.tensor([0, 10, 30, 40], dtype=torch.int32, device="cuda")
    smoe.smoe_experts_matmul_q8(x, one, R, order, 1, off, R, E, w, one, N, K, y, 0, wsp, need)
    assert smoe.smoe_last_device_status() == smoe.SMOE_ERR_ROUTE
    ref = torch.full((R, N), float(K), device="cuda")
    ref[3] = ref[20] = 0
    assert torch.equal(y, ref)
    order = torch.arange(R, dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 10, 1 << 30, 40], dtype=torch.int32, device="cuda")
    smoe.smoe_experts_matmul_q8(x, one, R, order, 1, off, R, E, w, one, N, K, y, 0, wsp, need)
    assert smoe.smoe_last_device_status() == smoe.SMOE_ERR_ROUTE
    assert torch.equal(y[:10], torch.full((10, N), float(K), device="cuda"))


@pytest.mark.parametrize("R", [1, 40, 400])
def test_weights_quantised_just_before_their_product(smoe, R):
    """The product's kernels start early; none may read weights that the
    quantiser in front of it is still writing."""
    N, K = 4096, 4096
    g = torch.Generator(device="cuda").manual_seed(R)
    x = torch.randn(R, K, generator=g, device="cuda")
    xq, xs = torch.empty(R, K, dtype=torch.int8, device="cuda"), torch.empty(R, device="cuda")
    wq, ws = torch.empty(N, K, dtype=torch.int8, device="cuda"), torch.empty(N, device="cuda")
    need = smoe.smoe_matmul_q8_workspace_bytes(R, N, K)
    wsp = torch.empty(need, dtype=torch.uint8, device="cuda")
    w = [torch.randn(N, K, generator=g, device="cuda") for _ in range(4)]
    y = [torch.empty(R, N, device="cuda") for _ in range(12)]
    smoe.smoe_quantize_rows_q8(x, 0, 0, R, K, xq, xs)
    torch.cuda.synchronize()
    for i, out in enumerate(y):
        smoe.smoe_quantize_rows_q8(w[i % 4], 0, 0, N, K, wq, ws)
        if i % 2:
            smoe.smoe_quantize_rows_q8(x, 0, 0, R, K, xq, xs)
        smoe.smoe_matmul_q8(xq, xs, R, wq, ws, N, K, out, 0, wsp, need)
    torch.cuda.synchronize()
    for i in range(4):
        smoe.smoe_quantize_rows_q8(w[i], 0, 0, N, K, wq, ws)
        torch.cuda.synchronize()
        smoe.smoe_matmul_q8(xq, xs, R, wq, ws, N, K, y[i], 0, wsp, need)
        torch.cuda.synchronize()
        for j in (4 + i, 8 + i):
            assert torch.equal(y[j], y[i])


@pytest.mark.parametrize("R", [40, 2000])
def test_experts_weights_past_32_bits(smoe, R):
    """4.4 GB of weights: the last expert's rows against float64."""
    E, N, K = 130, 8200, 4096
    wq = torch.zeros(E * N, K, dtype=torch.int8, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(R)
    last = torch.randint(-127, 128, (N, K), generator=g, device="cuda").to(torch.int8)
    wq[(E - 1) * N:] = last
    ws = torch.ones(E * N, device="cuda")
    xq = torch.randint(-127, 128, (R, K), generator=g, device="cuda").to(torch.int8)
    xs = torch.ones(R, device="cuda")
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[E] = R
    y = torch.empty(R, N, device="cuda")
    need = smoe.smoe_experts_matmul_q8_workspace_bytes(R, R, E, N, K)
    wsp = torch.empty(need, dtype=torch.uint8, device="cuda")
    smoe.smoe_experts_matmul_q8(xq, xs, R, None, 1, off, R, E, wq, ws, N, K, y, 0, wsp, need)
    torch.cuda.synchronize()
    ref = xq.double() @ last.double().t()
    mag = xq.double().abs() @ last.double().abs().t()
    assert ((y.double() - ref).abs() <= (K / 16 + 16) * U * mag).all()


def test_matmul_rows_past_32_bits(smoe):
    """Outputs past 4 GB."""
    R, N, K = 33000, 33000, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    xq = torch.randint(-127, 128, (R, K), generator=g, device="cuda").to(torch.int8)
    wq = torch.randint(-127, 128, (N, K), generator=g, device="cuda").to(torch.int8)
    one = torch.ones(R, device="cuda")
    y = torch.empty(R, N, device="cuda")
    need = smoe.smoe_matmul_q8_workspace_bytes(R, N, K)
    wsp = torch.empty(need, dtype=torch.uint8, device="cuda")
    smoe.smoe_matmul_q8(xq, one, R, wq, one, N, K, y, 0, wsp, need)
    torch.cuda.synchronize()
    for at in (0, R // 2, R - 100):
        ref = xq[at:at + 100].double() @ wq.double().t()
        assert torch.equal(y[at:at + 100].double(), ref)  # below 2^24: exact


def test_workspace_does_not_fall_as_the_batch_grows(smoe):
    for E in (1, 8, 128):
        last = 0
        for R in (1, 2, 3, 5, 40, 48, 49, 64, 65, 400, 5000, 6145, 20000):
            need = smoe.smoe_experts_matmul_q8_workspace_bytes(R, R, E, 256, 256)
            assert need >= last
            last = need
