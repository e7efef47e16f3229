"""8-bit floating-point quantisers and products on the GPU against float64 of the
same codes, and the codes against the float32 steps that define them."""
import numpy as np
import pytest

import f8_util as u

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch

    import moe_expert_ffn_smoe_gb300 as smoe
    return torch, smoe, torch.device("cuda:0")


def dtypes(torch, name):
    return (torch.bfloat16, 1) if name == "bf16" else (torch.float32, 0)


# ---------------------------------------------------------------- quantisers

def rows_f8(env, x, code, act, R, K):
    torch, smoe, dev = env
    q = torch.full((R, K), 0x55, dtype=torch.uint8, device=dev)
    s = torch.full((R, -(-K // 128)), -7.0, device=dev)
    smoe.smoe_quantize_rows_f8(x, code, act, R, K, q, s)
    return q.cpu().numpy(), s.cpu().numpy()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("R,K", [(1, 1), (3, 127), (2, 128), (5, 129), (33, 512), (7, 1000), (4, 1004), (65, 1544), (2, 32768),
                                 (1, 17)])
def test_rows_are_quantised_by_the_f32_steps(env, dtype, R, K):
    torch, smoe, dev = env
    dt, code = dtypes(torch, dtype)
    rng = np.random.default_rng([R, K])
    x = (rng.normal(size=(R, K)) * np.exp(3 * rng.normal(size=(R, 1)))).astype(np.float32)
    x[rng.random((R, K)) < 0.1] = 0
    X = torch.from_numpy(x).to(dev).to(dt)
    q, s = rows_f8(env, X, code, smoe.SMOE_Q8_PLAIN, R, K)
    rq, rs = u.quantize_rows(X.float().cpu().numpy())
    assert (s == rs).all() and (q == rq).all()


def test_rows_at_the_edges_of_f32(env):
    """Zeros, the smallest and largest numbers, NaN and infinities, each in one
    block of its row; a base that no vector fits."""
    torch, smoe, dev = env
    R, K = 9, 300
    rng = np.random.default_rng(4)
    x = rng.normal(size=(R, K)).astype(np.float32)
    x[0, :128] = 0
    x[1, 128:256] = rng.normal(size=128) * 1e-38
    x[2, 256:] = rng.integers(-9, 9, size=44) * np.float32(1e-45)
    x[3, :128] *= np.float32(1e38) / np.abs(x[3, :128]).max() * np.float32(3.4)
    x[4, 130] = np.nan
    x[5, 299] = np.inf
    x[6, 0] = -np.inf
    x[7, :128] = np.float32(1.4e-36) * rng.normal(size=128)
    x[8, :128] = 1
    buf = torch.empty(R * K + 1, device=dev)
    for at in (0, 1):
        X = buf[at:at + R * K].view(R, K)
        X.copy_(torch.from_numpy(x))
        q, s = rows_f8(env, X, 0, smoe.SMOE_Q8_PLAIN, R, K)
        rq, rs = u.quantize_rows(x)
        assert np.array_equal(s, rs, equal_nan=True) and (q == rq).all()
        assert np.isnan(s[[4, 5, 6], [1, 2, 0]]).all() and np.isnan(s).sum() == 3


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("R,K", [(3, 128), (17, 1536), (5, 200), (6, 77)])
def test_the_activation(env, dtype, R, K):
    torch, smoe, dev = env
    dt, code = dtypes(torch, dtype)
    rng = np.random.default_rng([R, K, 1])
    x = (rng.normal(size=(R, 2 * K)) * 4).astype(np.float32)
    x[0, :5] = [-100, -90, 90, 0, -0.0]
    X = torch.from_numpy(x).to(dev).to(dt)
    q, s = rows_f8(env, X, code, smoe.SMOE_Q8_SILU_MUL, R, K)
    v = X.double().cpu().numpy()
    v = v[:, :K] / (1 + np.exp(-v[:, :K])) * v[:, K:]
    top = np.stack([np.abs(v[:, c:c + 128]).max(1) for c in range(0, K, 128)], 1)
    # SiLU to 2^-20, three roundings
    assert (np.abs(s - top / 448) <= 2.0 ** -19 * top / 448).all()
    # a code: half a step of three mantissa bits, or of the smallest exponent
    assert (np.abs(u.rows_of(q, s) - v) <= (2.0 ** -4 + 2.0 ** -18) * np.abs(v) + u.spread(s, 1, K) * (2.0 ** -10 + 1e-6)).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,N,K,both", [(1, 128, 128, True), (3, 130, 257, True), (2, 64, 1000, True), (1, 1, 1, True),
                                        (2, 384, 132, False), (2, 129, 16, True), (5, 255, 383, True)])
def test_weights_are_quantised_in_blocks_both_ways(env, dtype, n, N, K, both):
    torch, smoe, dev = env
    dt, code = dtypes(torch, dtype)
    rng = np.random.default_rng([n, N, K])
    w = (rng.normal(size=(n, N, K)) * np.exp(rng.normal(size=(n, N, 1)))).astype(np.float32)
    w[0, :128, :128] *= 1e-37 if dtype == "f32" else 1
    W = torch.from_numpy(w).to(dev).to(dt)
    nb, kb = -(-N // 128), -(-K // 128)
    q, s = torch.full((n, N, K), 0x55, dtype=torch.uint8, device=dev), torch.full((n, nb, kb), -7.0, device=dev)
    qt, st = torch.full((n, K, N), 0x55, dtype=torch.uint8, device=dev), torch.full((n, kb, nb), -7.0, device=dev)
    smoe.smoe_quantize_blocks_f8(W, code, n, N, K, q, s, *((qt, st) if both else (None, None)))
    v, gq, gs = W.float().cpu().numpy(), q.cpu().numpy(), s.cpu().numpy()
    for m in range(n):
        for a in range(nb):
            for b in range(kb):
                at = (m, slice(a * 128, a * 128 + 128), slice(b * 128, b * 128 + 128))
                rq, rs = u.quantize(v[at])
                assert gs[m, a, b] == rs and (gq[at] == rq).all()
    if both:
        assert (qt.cpu().numpy() == gq.transpose(0, 2, 1)).all() and (st.cpu().numpy() == gs.transpose(0, 2, 1)).all()
    else:
        assert (qt.cpu().numpy() == 0x55).all() and (st.cpu().numpy() == -7).all()
    W[0, 0, 0] = float("nan")
    smoe.smoe_quantize_blocks_f8(W, code, n, N, K, q, s)
    assert np.isnan(s.cpu().numpy()).sum() == 1 and np.isnan(s[0, 0, 0].item())
    assert (q[0, :128, :128].cpu().numpy() == 0).all()


# ---------------------------------------------------------------- products

def codes(rng, *shape):
    """Codes over the whole type, finite."""
    return u.to_e4m3(np.clip(rng.normal(size=shape) * 100, -448, 448))


def bound(K, dtype, mag):
    """A sum of K exact products in 32 bits: 128 additions a block and one a block
    more, each off by at most 2^-23 of the magnitudes (a rounding towards zero; to
    nearest, half), the scales' product and its use; then the output's own type."""
    err = (128 + -(-K // 128) + 4) * 2.0 ** -23 * mag
    return err + (2.0 ** -8 * (mag + err) if dtype == "bf16" else 0) + 1e-37


def product(env, seed, R, N, K, dtype, n=1, offsets=None, order=None, k=1, nsrc=None, change=None):
    """(y, reference, magnitudes) of one call, whose buffers end in guard values."""
    torch, smoe, dev = env
    dt, code = dtypes(torch, dtype)
    rng = np.random.default_rng([seed, R, N, K, n])
    nsrc = nsrc or R
    kb, nb = -(-K // 128), -(-N // 128)
    xq, wq = codes(rng, nsrc, K), codes(rng, n, N, K)
    xs = rng.uniform(0.5, 2, size=(nsrc, kb)).astype(np.float32) * np.float32(2.0) ** rng.integers(-6, 6, size=(nsrc, kb))
    ws = rng.uniform(0.5, 2, size=(n, nb, kb)).astype(np.float32) * np.float32(2.0) ** rng.integers(-6, 6, size=(n, nb, kb))
    xs = xs.astype(np.float32)
    ws = ws.astype(np.float32)
    if change:
        change(xq, xs, wq, ws)
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    y = torch.full((R * N + 64,), 123.0, dtype=dt, device=dev)
    if offsets is None:
        need = smoe.smoe_matmul_f8_workspace_bytes(R, N, K)
        work = torch.empty(need, dtype=torch.uint8, device=dev)
        smoe.smoe_matmul_f8(d(xq), d(xs), R, d(wq), d(ws), N, K, y, code, work, need)
    else:
        need = smoe.smoe_experts_matmul_f8_workspace_bytes(nsrc, R, n, N, K)
        work = torch.empty(need, dtype=torch.uint8, device=dev)
        smoe.smoe_experts_matmul_f8(d(xq), d(xs), nsrc, None if order is None else d(order.astype(np.int32)), k,
                                    d(np.asarray(offsets, np.int32)), R, n, d(wq), d(ws), N, K, y, code, work, need)
    assert smoe.smoe_last_device_status() == smoe.SMOE_OK
    assert (y[R * N:].float() == 123).all()
    x, w = d(u.rows_of(xq, xs)), d(u.weights_of(wq, ws))
    ref, mag = torch.zeros(R, N, dtype=torch.float64, device=dev), torch.zeros(R, N, dtype=torch.float64, device=dev)
    at = [0, R] if offsets is None else offsets
    for e in range(n):
        a, b = at[e], at[e + 1]
        if b > a:
            rows = x[a:b] if order is None else x[d(order[a:b] // k)]
            ref[a:b], mag[a:b] = rows @ w[e].t(), rows.abs() @ w[e].abs().t()
    return y[:R * N].view(R, N).double(), ref, mag


def hold(torch, got, K, dtype):
    y, ref, mag = got
    worst = ((y - ref).abs() / bound(K, dtype, mag)).max().item()
    assert worst <= 1, worst


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("R,N,K", [(1, 1, 16), (1, 100, 128), (2, 129, 1040), (1, 1000, 4096), (3, 7, 16), (3, 128, 4096), (4, 136, 144),
                                   (16, 512, 512), (17, 257, 2064), (63, 384, 1024), (65, 130, 272), (100, 1024, 2048),
                                   (300, 1000, 1024), (1025, 514, 400), (700, 2056, 4096), (2049, 1536, 640)])
def test_one_matrix(env, dtype, R, N, K):
    hold(env[0], product(env, 1, R, N, K, dtype), K, dtype)


def batch(rng, n, counts, tail, k):
    """offsets, order, sources of a batch of those counts and `tail` rows of none."""
    R = int(sum(counts)) + tail
    R += -R % k
    order = rng.permutation(R)
    return np.concatenate([[0], np.cumsum(counts)]), order, R, R // k


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("n,counts,tail,N,K", [
    (4, [1, 0, 1, 0], 0, 100, 160), (8, [0, 0, 0, 1, 0, 0, 0, 0], 3, 130, 256), (3, [5, 0, 20], 1, 257, 400),
    (5, [64, 65, 0, 1, 130], 6, 384, 1024), (2, [0, 0], 40, 128, 128), (6, [300, 17, 0, 256, 511, 33], 9, 520, 912),
    (16, [2] * 16, 0, 512, 2048), (40, [0, 9] * 20, 5, 136, 384), (3, [1000, 0, 700], 2, 200, 272)])
def test_experts(env, dtype, gather, n, counts, tail, N, K):
    rng = np.random.default_rng([n, N, K])
    offsets, order, R, nsrc = batch(rng, n, counts, tail, 2 if gather else 1)
    got = product(env, 2, R, N, K, dtype, n, offsets.tolist(), order if gather else None, 2 if gather else 1, nsrc)
    hold(env[0], got, K, dtype)
    assert (got[0][int(offsets[-1]):] == 0).all()  # rows of no expert


@pytest.mark.parametrize("R,experts", [(1, False), (40, False), (700, False), (300, True)])
def test_nan_codes_and_scales_reach_their_outputs_alone(env, R, experts):
    torch = env[0]
    N, K, n = 300, 528, 2 if experts else 1
    offsets = [0, R // 3, R] if experts else None

    def change(xq, xs, wq, ws):
        xq[R // 2, 7] = 0x7f
        if R > 1:
            xs[R - 1, 4] = np.nan
        wq[n - 1, 131, 300] = 0xff
        ws[n - 1, 2, 1] = np.nan  # outputs 256 to 299

    y, ref, mag = product(env, 3, R, N, K, "f32", n, offsets, change=change)
    assert (torch.isnan(y) == torch.isnan(ref)).all()
    fine = ~torch.isnan(ref)
    assert 0 < fine.sum() < fine.numel() or R == 1
    assert ((y - ref).abs()[fine] <= bound(K, "f32", mag)[fine]).all()


def test_more_weights_than_32_bits_count(env):
    """An expert whose matrix begins past 2^32 bytes, and rows past 2^31 outputs'
    bytes are addressed in 64 bits."""
    torch, smoe, dev = env
    n, N, K, R = 70, 2048, 32768, 40
    need = smoe.smoe_experts_matmul_f8_workspace_bytes(R, R, n, N, K)
    wq = torch.zeros(n, N, K, dtype=torch.uint8, device=dev)  # 4.7 GB
    wq[n - 1, :, -16:] = 0x38  # ones
    ws, xs = torch.ones(n, 16, 256, device=dev), torch.ones(R, 256, device=dev)
    xq = torch.full((R, K), 0x40, dtype=torch.uint8, device=dev)  # twos
    for rows in (R, 2):
        off = torch.zeros(n + 1, dtype=torch.int32, device=dev)
        off[n] = rows
        y = torch.empty(rows, N, device=dev)
        smoe.smoe_experts_matmul_f8(xq, xs, R, None, 1, off, rows, n, wq, ws, N, K, y, smoe.SMOE_F32,
                                    torch.empty(need, dtype=torch.uint8, device=dev), need)
        assert (y == 32).all()
    assert smoe.smoe_last_device_status() == smoe.SMOE_OK


@pytest.mark.parametrize("R", [3, 200])
def test_lists_that_are_none_are_reported(env, R):
    """Offsets that do not ascend or leave the rows, an order that points outside:
    reported, and nothing outside the outputs is written."""
    torch, smoe, dev = env
    n, N, K = 4, 136, 256
    rng = np.random.default_rng(0)
    xq, wq = torch.from_numpy(codes(rng, R, K)).to(dev), torch.from_numpy(codes(rng, n, N, K)).to(dev)
    xs, ws = torch.ones(R, 2, device=dev), torch.ones(n, 2, 2, device=dev)
    need = smoe.smoe_experts_matmul_f8_workspace_bytes(R, R, n, N, K)
    work = torch.empty(need, dtype=torch.uint8, device=dev)
    order = torch.arange(R, dtype=torch.int32, device=dev)
    for off, bad in (([0, 2, 1, 2, R], None), ([-5, 0, 1, 2, R], None), ([0, 1, 2, R + 9, R], None), ([0, 1, 1, 2, R], 1 << 30),
                     ([0, 1, 1, 2, R], -1), ([0, 1, 1, 2, R], R)):
        o = order.clone()
        if bad is not None:
            o[R - 1] = bad
        y = torch.full((R * N + 64,), 5.0, device=dev)
        smoe.smoe_experts_matmul_f8(xq, xs, R, o, 1, torch.tensor(off, dtype=torch.int32, device=dev), R, n, wq, ws, N, K, y,
                                    smoe.SMOE_F32, work, need)
        assert smoe.smoe_last_device_status() == smoe.SMOE_ERR_ROUTE
        assert (y[R * N:] == 5).all()
        if bad is not None:
            assert (y.view(-1)[(R - 1) * N:R * N] == 0).all()  # no source: zeros
    y = torch.full((R * N,), 5.0, device=dev)
    smoe.smoe_experts_matmul_f8(xq, xs, R, order, 1, torch.tensor([0, 1, 1, 2, R], dtype=torch.int32, device=dev), R, n, wq, ws,
                                N, K, y, smoe.SMOE_F32, work, need)
    assert smoe.smoe_last_device_status() == smoe.SMOE_OK


def test_the_input_gradient_and_a_graph_on_another_stream(env):
    """Rows quantised, multiplied by the weights and by the transposed ones that the
    quantiser made, all captured in one graph and replayed on new inputs."""
    torch, smoe, dev = env
    n, N, K, R = 6, 320, 528, 333
    g = torch.Generator(device=dev).manual_seed(0)
    w = torch.randn(n, N, K, generator=g, device=dev)
    x, dy = torch.empty(R, K, device=dev), torch.empty(R, N, dtype=torch.bfloat16, device=dev)
    off = torch.tensor([0, 10, 10, 100, 101, 290, 330], dtype=torch.int32, device=dev)
    u8 = lambda *s: torch.empty(*s, dtype=torch.uint8, device=dev)  # noqa: E731
    f32 = lambda *s: torch.empty(*s, device=dev)  # noqa: E731
    q, qt, s, st = u8(n, N, K), u8(n, K, N), f32(n, 3, 5), f32(n, 5, 3)
    xq, xs, dq, ds = u8(R, K), f32(R, 5), u8(R, N), f32(R, 3)
    y, dx = f32(R, N), f32(R, K)
    need = smoe.smoe_experts_matmul_f8_workspace_bytes(R, R, n, max(N, K), max(N, K))
    work, stream = u8(need), torch.cuda.Stream()

    def calls():
        smoe.smoe_quantize_blocks_f8(w, smoe.SMOE_F32, n, N, K, q, s, qt, st, stream)
        smoe.smoe_quantize_rows_f8(x, smoe.SMOE_F32, smoe.SMOE_Q8_PLAIN, R, K, xq, xs, stream)
        smoe.smoe_experts_matmul_f8(xq, xs, R, None, 1, off, R, n, q, s, N, K, y, smoe.SMOE_F32, work, need, stream)
        smoe.smoe_quantize_rows_f8(dy, smoe.SMOE_BF16, smoe.SMOE_Q8_PLAIN, R, N, dq, ds, stream)
        smoe.smoe_experts_matmul_f8(dq, ds, R, None, 1, off, R, n, qt, st, K, N, dx, smoe.SMOE_F32, work, need, stream)

    x.normal_(generator=g)
    dy.normal_(generator=g)
    torch.cuda.synchronize()
    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        calls()
    for _ in range(2):
        x.normal_(generator=g)
        dy.normal_(generator=g)
        w.normal_(generator=g)
        graph.replay()
        torch.cuda.synchronize()
        d = lambda a: torch.from_numpy(a).to(dev)  # noqa: E731
        W = d(u.weights_of(q.cpu().numpy(), s.cpu().numpy()))
        X, DY = d(u.rows_of(xq.cpu().numpy(), xs.cpu().numpy())), d(u.rows_of(dq.cpu().numpy(), ds.cpu().numpy()))
        for got, rows, mats, width in ((y, X, W.transpose(1, 2), K), (dx, DY, W, N)):
            for e in range(n):
                a, b = off[e].item(), off[e + 1].item()
                mag = rows[a:b].abs() @ mats[e].abs()
                assert ((got[a:b] - rows[a:b] @ mats[e]).abs() <= bound(width, "f32", mag)).all()
            assert (got[330:] == 0).all()
    assert smoe.smoe_last_device_status() == smoe.SMOE_OK


def test_the_same_inputs_give_the_same_bits(env):
    torch, smoe, dev = env
    for R, N, K in ((1, 1000, 2048), (20, 512, 4096), (900, 1000, 1024)):
        a, b = product(env, 7, R, N, K, "f32")[0], product(env, 7, R, N, K, "f32")[0]
        assert (a == b).all()


# ---------------------------------------------------------------- large batches: the rows on the other side of the product

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("R,N,K", [(1500, 2049, 1040), (1999, 4096, 512), (640, 8200, 16), (1100, 4000, 4240)])
def test_one_matrix_and_many_rows(env, dtype, R, N, K):
    hold(env[0], product(env, 8, R, N, K, dtype), K, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("n,counts,tail,N,K", [
    (6, [300, 17, 0, 256, 511, 33], 9, 4104, 272), (3, [1000, 0, 701], 3, 4097, 144), (40, [0, 90] * 20, 5, 2500, 1040),
    (9, [128, 129, 127, 1, 0, 255, 257, 383, 4], 700, 4000, 640), (2, [0, 0], 1500, 4100, 128)])
def test_experts_and_many_rows(env, dtype, gather, n, counts, tail, N, K):
    rng = np.random.default_rng([n, N, K])
    offsets, order, R, nsrc = batch(rng, n, counts, tail, 3 if gather else 1)
    got = product(env, 9, R, N, K, dtype, n, offsets.tolist(), order if gather else None, 3 if gather else 1, nsrc)
    hold(env[0], got, K, dtype)
    assert (got[0][int(offsets[-1]):] == 0).all()  # rows of no expert


@pytest.mark.parametrize("gather", [True, False])
def test_nan_reaches_its_outputs_alone_among_many_rows(env, gather):
    """NaN codes and scales of rows and weights, in the middle of a tile and at its
    edges, and in rows that no expert has."""
    torch = env[0]
    N, K, n, R = 4100, 272, 2, 1207
    offsets = [0, 500, 1200]
    order = np.random.default_rng(2).permutation(R) if gather else np.arange(R)

    def change(xq, xs, wq, ws):
        xq[order[127], 7] = 0x7f
        xs[order[500], 1] = np.nan
        xq[order[1199], 271] = 0xff
        xq[order[1204]] = 0x7f  # behind the last expert
        wq[1, 131, 200] = 0xff
        ws[1, 32, 2] = np.nan  # outputs 4096 to 4099

    y, ref, mag = product(env, 10, R, N, K, "f32", n, offsets, order if gather else None, 1, change=change)
    ref[1200:] = 0
    assert (torch.isnan(y) == torch.isnan(ref)).all()
    fine = ~torch.isnan(ref)
    assert ((y - ref).abs()[fine] <= bound(K, "f32", mag)[fine]).all()


def test_lists_that_are_none_are_reported_for_many_rows(env):
    torch, smoe, dev = env
    n, N, K, R = 4, 4104, 256, 1500
    rng = np.random.default_rng(0)
    xq, wq = torch.from_numpy(codes(rng, R, K)).to(dev), torch.from_numpy(codes(rng, n, N, K)).to(dev)
    xs, ws = torch.ones(R, 2, device=dev), torch.ones(n, 33, 2, device=dev)
    need = smoe.smoe_experts_matmul_f8_workspace_bytes(R, R, n, N, K)
    work = torch.empty(need, dtype=torch.uint8, device=dev)
    order = torch.arange(R, dtype=torch.int32, device=dev)
    for off, bad in (([0, 900, 700, 1400, R], None), ([-5, 0, 700, 1400, R], None), ([0, 500, 700, R + 9, R], None),
                     ([0, 500, 500, 600, R], 1 << 30), ([0, 500, 500, 600, R], -1), ([0, 500, 500, 600, R], R)):
        o = order.clone()
        if bad is not None:
            o[R - 1] = bad
        y = torch.full((R * N + 64,), 5.0, device=dev)
        smoe.smoe_experts_matmul_f8(xq, xs, R, o, 1, torch.tensor(off, dtype=torch.int32, device=dev), R, n, wq, ws, N, K, y,
                                    smoe.SMOE_F32, work, need)
        assert smoe.smoe_last_device_status() == smoe.SMOE_ERR_ROUTE
        assert (y[R * N:] == 5).all()
        if bad is not None:
            assert (y.view(-1)[(R - 1) * N:R * N] == 0).all()  # no source: zeros


def test_scales_at_odd_addresses_among_many_rows(env):
    """The row scales' vectors of four where they begin at no 16-byte boundary."""
    torch, smoe, dev = env
    R, N, K = 1300, 2100, 512
    g = torch.Generator(device=dev).manual_seed(0)
    x, w = torch.randn(R, K, generator=g, device=dev), torch.randn(1, N, K, generator=g, device=dev)
    u8 = lambda *s: torch.empty(*s, dtype=torch.uint8, device=dev)  # noqa: E731
    xq, xs, wq, ws = u8(R, K), torch.empty(R, 4, device=dev), u8(1, N, K), torch.empty(1, 17, 4, device=dev)
    smoe.smoe_quantize_rows_f8(x, smoe.SMOE_F32, smoe.SMOE_Q8_PLAIN, R, K, xq, xs)
    smoe.smoe_quantize_blocks_f8(w, smoe.SMOE_F32, 1, N, K, wq, ws)
    odd_x, odd_w = torch.empty(R * 4 + 1, device=dev), torch.empty(17 * 4 + 1, device=dev)
    odd_x[1:], odd_w[1:] = xs.view(-1), ws.view(-1)
    ys = []
    need = smoe.smoe_matmul_f8_workspace_bytes(R, N, K)
    for a, b in ((xs, ws), (odd_x[1:], odd_w[1:])):
        ys.append(torch.full((R, N), float("nan"), device=dev))
        smoe.smoe_matmul_f8(xq, a, R, wq, b, N, K, ys[-1], smoe.SMOE_F32, u8(need), need)
    assert torch.equal(*ys) and smoe.smoe_last_device_status() == smoe.SMOE_OK


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sums_of_nothing(env, dtype):
    torch, smoe, dev = env
    dt, code = dtypes(torch, dtype)
    R, N = 37, 101
    one = torch.zeros(16, dtype=torch.uint8, device=dev)
    f = torch.zeros(16, device=dev)
    y = torch.full((R * N + 8,), 3.0, dtype=dt, device=dev)
    need = smoe.smoe_matmul_f8_workspace_bytes(R, N, 0)
    smoe.smoe_matmul_f8(one, f, R, one, f, N, 0, y, code, torch.empty(max(need, 16), dtype=torch.uint8, device=dev), need)
    assert (y[:R * N] == 0).all() and (y[R * N:] == 3).all()


def test_many_rows_at_once_on_two_streams(env):
    """Two products with workspaces of their own, started together again and again."""
    torch, smoe, dev = env
    n, N, K, R = 8, 4000, 512, 1800
    g = torch.Generator(device=dev).manual_seed(1)
    u8 = lambda *s: torch.empty(*s, dtype=torch.uint8, device=dev)  # noqa: E731
    need = smoe.smoe_experts_matmul_f8_workspace_bytes(R, R, n, N, K)
    calls, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for off in ([0, 200, 200, 500, 900, 901, 1300, 1700, 1790], [0, 1000, 1100, 1200, 1300, 1400, 1500, 1600, 1800]):
        x, w = torch.randn(R, K, generator=g, device=dev), torch.randn(n, N, K, generator=g, device=dev)
        xq, xs, wq, ws = u8(R, K), torch.empty(R, 4, device=dev), u8(n, N, K), torch.empty(n, 32, 4, device=dev)
        smoe.smoe_quantize_rows_f8(x, smoe.SMOE_F32, smoe.SMOE_Q8_PLAIN, R, K, xq, xs)
        smoe.smoe_quantize_blocks_f8(w, smoe.SMOE_F32, n, N, K, wq, ws)
        calls.append((xq, xs, R, None, 1, torch.tensor(off, dtype=torch.int32, device=dev), R, n, wq, ws, N, K))
    run = lambda c, y, ws, s: smoe.smoe_experts_matmul_f8(*c, y, smoe.SMOE_F32, ws, need, s)  # noqa: E731
    alone, outs = ([torch.empty(R, N, device=dev) for _ in range(2)] for _ in range(2))
    work = [u8(need) for _ in range(2)]
    for c, y in zip(calls, alone):
        run(c, y, work[0], None)
    torch.cuda.synchronize()
    for _ in range(10):
        for c, y, ws, s in zip(calls, outs, work, streams):
            run(c, y, ws, s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(alone, outs)) and smoe.smoe_last_device_status() == smoe.SMOE_OK
