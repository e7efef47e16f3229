"""The gradient of the experts' weights on the GPU against float64."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch

    import moe_expert_ffn_smoe_gb300 as smoe
    return torch, smoe, torch.device("cuda:0")


def grad(env, seed, counts, tail, N, K, dtype, before=None, change=None):
    """(d_w, reference, magnitudes, rows of each expert)."""
    torch, smoe, dev = env
    g = torch.Generator(device=dev).manual_seed(seed)
    n, R = len(counts), int(sum(counts)) + tail
    at = np.concatenate([[0], np.cumsum(counts)]).tolist()
    dy = torch.randn(R, N, generator=g, device=dev).to(torch.bfloat16)
    x = torch.randn(R, K, generator=g, device=dev).to(torch.bfloat16)
    if change:
        change(dy, x, at)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    out = torch.full((n * N * K + 64,), 77.0, dtype=dt, device=dev)
    if before is not None:
        out[:n * N * K] = before.reshape(-1)
    smoe.smoe_experts_weight_grad(dy, x, torch.tensor(at, dtype=torch.int32, device=dev), R, n, N, K, int(before is not None),
                                  out, 1 if dtype == "bf16" else 0)
    assert smoe.smoe_last_device_status() == smoe.SMOE_OK
    assert (out[n * N * K:] == 77).all()
    ref, mag = [], []
    for a, b in zip(at[:-1], at[1:]):
        ref.append(dy[a:b].double().t() @ x[a:b].double())
        mag.append(dy[a:b].double().abs().t() @ x[a:b].double().abs())
    return out[:n * N * K].view(n, N, K).double(), torch.stack(ref), torch.stack(mag), np.asarray(counts)


def hold(got, dtype, more=0.0):
    """A sum of an expert's rows in 32 bits, each addition off by at most 2^-23 of
    the magnitudes (a rounding towards zero), and the output's own type."""
    d, ref, mag, counts = got
    for e, c in enumerate(counts):
        err = (c + 2) * 2.0 ** -23 * mag[e]
        b = err + (2.0 ** -8 * (ref[e].abs() + err) if dtype == "bf16" else 2.0 ** -24 * ref[e].abs()) + more
        assert ((d[e] - ref[e]).abs() <= b + 1e-37).all(), (e, c)
        if c == 0:
            assert (d[e] == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("counts,tail,N,K", [
    ([1], 0, 8, 8), ([0], 5, 16, 24), ([0, 3, 0], 0, 128, 256), ([8, 9, 15, 16, 17], 4, 72, 264), ([64, 63, 65, 128, 1], 0, 256, 256),
    ([7, 0, 200, 31], 3, 264, 520), ([1000, 2, 0, 500], 11, 136, 1032), ([33] * 20, 0, 520, 136), ([5000], 0, 128, 64),
    ([2, 0, 1] * 30, 0, 768, 512)])
def test_weight_gradient(env, dtype, counts, tail, N, K):
    hold(grad(env, 1, counts, tail, N, K, dtype), dtype)


def test_rows_of_others_never_meet_an_experts_sum(env):
    """NaN and infinities in the rows just before and after an expert's, and past
    the last one's: its own gradient stays finite."""
    def change(dy, x, at):
        for e in (0, 2, 4):
            dy[at[e]:at[e + 1]] = float("nan")
            x[at[e]:at[e + 1]] = float("inf")
        dy[at[-1]:] = float("nan")
        x[at[-1]:] = float("nan")

    for odd in (1, 5, 13, 16, 30, 64, 71):
        d, ref, mag, counts = grad(env, odd, [3, odd, 9, odd + 2, 20, odd], 6, 136, 264, "f32", change=change)
        fine = [1, 3, 5]
        assert d[fine].isfinite().all() and not d[[0, 2, 4]].isfinite().any()
        hold((d[fine], ref[fine], mag[fine], counts[fine]), "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_accumulation(env, dtype):
    torch, smoe, dev = env
    counts, N, K = [20, 0, 77], 136, 264
    before = (torch.arange(3 * N * K, device=dev) % 61 - 30).float().view(3, N, K)
    d, ref, mag, c = grad(env, 3, counts, 2, N, K, dtype, before=before)
    total = ref + before.double()
    step = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    for e in range(3):
        err = (c[e] + 2) * 2.0 ** -23 * mag[e]
        first = err + step * (ref[e].abs() + err)  # the sum, rounded
        assert ((d[e] - total[e]).abs() <= first + step * (total[e].abs() + first)).all()
    assert (d[1] == before[1]).all()


def test_it_is_the_gradient_of_the_product(env):
    """Against differences of sum(dy * (x w^T)) in w, in float64 on the same rows: the
    form is linear in w, so differences are exact but for 2^-53."""
    torch, smoe, dev = env
    d, ref, mag, c = grad(env, 5, [6, 11], 0, 16, 24, "f32")
    g = torch.Generator(device=dev).manual_seed(5)
    dy = torch.randn(17, 16, generator=g, device=dev).to(torch.bfloat16).double()
    x = torch.randn(17, 24, generator=g, device=dev).to(torch.bfloat16).double()
    loss = lambda w: sum((dy[a:b] * (x[a:b] @ w[e].t())).sum() for e, (a, b) in enumerate([(0, 6), (6, 17)]))  # noqa: E731
    w = torch.zeros(2, 16, 24, dtype=torch.float64, device=dev)
    for e, i, j in ((0, 0, 0), (0, 15, 23), (1, 3, 17), (1, 9, 8)):
        p, m = w.clone(), w.clone()
        p[e, i, j], m[e, i, j] = 1, -1
        assert abs((loss(p) - loss(m)) / 2 - d[e, i, j]) <= 2.0 ** -19 * mag[e, i, j]


def test_lists_that_are_none_no_rows_and_a_graph(env):
    torch, smoe, dev = env
    n, N, K, R = 3, 64, 72, 50
    dy, x = torch.ones(R, N, dtype=torch.bfloat16, device=dev), torch.ones(R, K, dtype=torch.bfloat16, device=dev)
    out = torch.full((n, N, K), 9.0, device=dev)
    for off in ([0, 30, 20, 50], [-1, 3, 4, 50], [0, 3, 4, 51]):
        smoe.smoe_experts_weight_grad(dy, x, torch.tensor(off, dtype=torch.int32, device=dev), R, n, N, K, 0, out, 0)
        assert smoe.smoe_last_device_status() == smoe.SMOE_ERR_ROUTE
    smoe.smoe_experts_weight_grad(None, None, torch.zeros(n + 1, dtype=torch.int32, device=dev), 0, n, N, K, 0, out, 0)
    assert (out == 0).all()
    off, s = torch.tensor([0, 10, 10, 50], dtype=torch.int32, device=dev), torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        smoe.smoe_experts_weight_grad(dy, x, off, R, n, N, K, 1, out, 0, s)
    g.replay()
    off.copy_(torch.tensor([0, 0, 50, 50]))
    g.replay()
    torch.cuda.synchronize()
    assert (out == torch.tensor([10.0, 50.0, 40.0], device=dev)[:, None, None]).all()
    assert smoe.smoe_last_device_status() == smoe.SMOE_OK
