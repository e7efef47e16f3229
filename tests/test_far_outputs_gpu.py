"""Outputs past 2^31 and 2^32 bytes, of the 8-bit floating-point product in both its forms and of
the weights' gradient; offsets that are none in the weights' gradient, expert by expert."""
import numpy as np
import pytest

import f8_util as u

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def smoe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build_library()
    import moe_expert_ffn_smoe_gb300 as m
    return m


def codes(rng, *shape):
    return u.to_e4m3(np.clip(rng.normal(size=shape) * 100, -448, 448))


def product(smoe, R, N, K, n, gather, dt):
    """y of R rows, its last 64 elements guards; and what its rows are sums of."""
    rng = np.random.default_rng([R, N, n])
    src = 997  # rows of xq, each many times (sorted: a pattern that repeats)
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    kb, nb = -(-K // 128), -(-N // 128)
    xq, xs = codes(rng, src, K), rng.uniform(0.5, 2, (src, kb)).astype(np.float32)
    wq, ws = codes(rng, n, N, K), rng.uniform(0.5, 2, (n, nb, kb)).astype(np.float32)
    row = torch.arange(R, device="cuda") * 389 % src
    off = torch.tensor([R * e // n for e in range(n)] + [R - 5], dtype=torch.int32, device="cuda")
    y = torch.full((R * N + 64,), 123.0, dtype=dt, device="cuda")
    need = smoe.smoe_experts_matmul_f8_workspace_bytes(src if gather else R, R, n, N, K)
    work = torch.empty(need, dtype=torch.uint8, device="cuda")
    rows, scales, order = (d(xq), d(xs), row.int()) if gather else (d(xq)[row], d(xs)[row], None)
    smoe.smoe_experts_matmul_f8(rows, scales, src if gather else R, order, 1, off, R, n, d(wq), d(ws), N, K, y,
                                int(dt == torch.bfloat16), work, need)
    assert smoe.smoe_last_device_status() == smoe.SMOE_OK
    assert (y[R * N:] == 123).all()
    return y[:R * N].view(R, N), d(u.rows_of(xq, xs)), d(u.weights_of(wq, ws)), row, off.tolist()


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("R,N,n,dt", [(600_011, 4096, 3, torch.bfloat16), (300_007, 4100, 2, torch.float32),
                                      (9_000_011, 128, 2, torch.float32), (6_000_001, 100, 3, torch.float32)])
def test_rows_of_products(smoe, R, N, n, dt, gather):
    """The first rows, those where the bytes before them reach 2^31 and 2^32, the last."""
    K = 16
    y, x, w, row, at = product(smoe, R, N, K, n, gather, dt)
    e = y.element_size()
    for edge in (0, at[1], 2 ** 31 // (N * e), 2 ** 32 // (N * e), R - 200):
        lo, hi = max(0, edge - 200), min(R, edge + 200)
        if lo >= hi:
            continue
        for m in range(n):
            a, b = max(lo, at[m]), min(hi, at[m + 1])
            if a >= b:
                continue
            ref, mag = x[row[a:b]] @ w[m].t(), x[row[a:b]].abs() @ w[m].abs().t()
            # 16 products in f32 (steps of 2^-23), two scales; the type's rounding
            err = 21 * 2.0 ** -23 * mag
            bound = err + (2.0 ** -8 * (ref.abs() + err) if dt == torch.bfloat16 else 0)
            assert ((y[a:b].double() - ref).abs() <= bound).all(), (m, a, b)
    assert (y[at[n]:] == 0).all()  # rows of no expert
    # every row was written: the sum of all against that of the patterns' sums
    some = torch.randint(0, at[n], (20_000,), device="cuda", generator=torch.Generator(device="cuda").manual_seed(0))
    expert = torch.bucketize(some, torch.tensor(at[1:n], device="cuda"), right=True)
    got = y[some].double().sum(1)
    ref, mag = torch.zeros(len(some), dtype=torch.float64, device="cuda"), torch.zeros(len(some), dtype=torch.float64, device="cuda")
    for m in range(n):
        mine = expert == m
        ref[mine] = x[row[some[mine]]] @ w[m].sum(0)
        mag[mine] = x[row[some[mine]]].abs() @ w[m].abs().sum(0)
    assert ((got - ref).abs() <= (21 * 2.0 ** -23 + (2.0 ** -7 if dt == torch.bfloat16 else 0)) * mag).all()


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_gradients_of_weights(smoe, dt):
    """The last expert's matrix begins past 2^32 bytes; added to, it keeps what was there."""
    N, K, counts = 2056, 4104, [3, 0, 70, 1] * 33 + [17]
    n, R = len(counts), int(np.sum(counts)) + 2
    at = [0, *np.cumsum(counts).tolist()]
    g = torch.Generator(device="cuda").manual_seed(1)
    dy = torch.randn(R, N, generator=g, device="cuda").to(torch.bfloat16)
    x = torch.randn(R, K, generator=g, device="cuda").to(torch.bfloat16)
    out = torch.full((n * N * K + 64,), 77.0, dtype=dt, device="cuda")
    off = torch.tensor(at, dtype=torch.int32, device="cuda")
    code = int(dt == torch.bfloat16)
    step = 2.0 ** -8 if dt == torch.bfloat16 else 2.0 ** -24
    for add in (0, 1):
        smoe.smoe_experts_weight_grad(dy, x, off, R, n, N, K, add, out, code)
        assert smoe.smoe_last_device_status() == smoe.SMOE_OK and (out[n * N * K:] == 77).all()
        d = out[:n * N * K].view(n, N, K)
        for e in (0, 1, 2, 63, 64, 65, 66, n - 3, n - 2, n - 1):
            a, b = dy[at[e]:at[e + 1]].double(), x[at[e]:at[e + 1]].double()
            ref, mag = a.t() @ b, a.abs().t() @ b.abs()
            err = (counts[e] + 2) * 2.0 ** -23 * mag
            err = err + step * (ref.abs() + err)
            if add:  # the same sum again, rounded once more
                ref, err = 2 * ref, 2 * err + step * (2 * ref.abs() + 2 * err)
            assert ((d[e].double() - ref).abs() <= err + 1e-37).all(), e


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("off,bad", [([0, 30, 20, 50], [1]), ([-1, 3, 4, 50], [0]), ([0, 3, 4, 51], [2]), ([0, -5, 60, 50], [0, 1, 2]),
                                     ([1 << 30, 7, 9, -(1 << 31)], [0, 2])])
def test_ranges_that_are_none(smoe, dt, off, bad):
    """A range that does not ascend or leaves the rows counts as empty and is reported;
    the others' sums stand, and nothing is written outside the matrices."""
    n, N, K, R = 3, 136, 264, 50
    g = torch.Generator(device="cuda").manual_seed(2)
    # whole numbers: sums of products are exact in both types' f32, and below 2^8 in bf16
    dy = torch.randint(-1, 2, (R, N), generator=g, device="cuda").to(torch.bfloat16)
    x = torch.randint(-1, 2, (R, K), generator=g, device="cuda").to(torch.bfloat16)
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    for add in (0, 1):
        buf = torch.full((64 + n * N * K + 64,), 5.0, dtype=dt, device="cuda")
        smoe.smoe_experts_weight_grad(dy, x, offsets, R, n, N, K, add, buf[64:], int(dt == torch.bfloat16))
        assert smoe.smoe_last_device_status() == smoe.SMOE_ERR_ROUTE
        assert (buf[:64] == 5).all() and (buf[64 + n * N * K:] == 5).all()
        d = buf[64:64 + n * N * K].view(n, N, K)
        for e in range(n):
            lo, hi = (0, 0) if e in bad else (off[e], off[e + 1])
            want = dy[lo:hi].float().t() @ x[lo:hi].float() + (5 if add else 0)
            assert torch.equal(d[e].float(), want), e
