"""Blocks of zeros in the 8-bit floating-point quantisers: scale 0, and codes that keep
the sign of their zero; their products are 0."""
import numpy as np
import pytest

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


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_blocks_of_zeros(smoe, dt):
    R, K, N = 3, 384, 256
    x, w = torch.ones(R, K, device="cuda"), torch.ones(1, N, K, device="cuda")
    x[:, 128:256] = 0.0
    x[1, 128:256:3] = -0.0
    x[2] = -0.0
    w[0, :128, :128], w[0, :128, 1] = 0.0, -0.0
    u8 = lambda *s: torch.full(s, 0x55, dtype=torch.uint8, device="cuda")  # noqa: E731
    xq, xs, wq, ws = u8(R, K), torch.full((R, 3), 7.0, device="cuda"), u8(1, N, K), torch.full((1, 2, 3), 7.0, device="cuda")
    qt, st = u8(1, K, N), torch.full((1, 3, 2), 7.0, device="cuda")
    code = int(dt == torch.bfloat16)
    smoe.smoe_quantize_rows_f8(x.to(dt), code, smoe.SMOE_Q8_PLAIN, R, K, xq, xs)
    smoe.smoe_quantize_blocks_f8(w.to(dt), code, 1, N, K, wq, ws, qt, st)
    sign = lambda t: torch.where(torch.signbit(t), 0x80, 0)  # noqa: E731
    assert (xs[:, 1] == 0).all() and (xs[2] == 0).all() and (xs[:2, [0, 2]] > 0).all()
    assert torch.equal(xq[:, 128:256].int(), sign(x[:, 128:256])) and torch.equal(xq[2].int(), sign(x[2]))
    assert ws[0, 0, 0] == 0 and (ws.view(-1)[1:] > 0).all() and torch.equal(st, ws.transpose(1, 2))
    assert torch.equal(wq[0, :128, :128].int(), sign(w[0, :128, :128])) and torch.equal(qt, wq.transpose(1, 2))
    need = smoe.smoe_matmul_f8_workspace_bytes(R, N, K)
    y = torch.full((R, N), float("nan"), device="cuda")
    smoe.smoe_matmul_f8(xq, xs, R, wq, ws, N, K, y, smoe.SMOE_F32, torch.empty(need, dtype=torch.uint8, device="cuda"), need)
    ones = xs[0, 0].item() * 448
    want = torch.tensor([[128.0, 256.0]] * 2 + [[0.0, 0.0]], device="cuda").repeat_interleave(128, 1) * ones * ones
    # two blocks of 128 products in f32, each addition off by 2^-23 at most, two scales
    assert ((y - want).abs() <= 260 * 2.0 ** -23 * want).all()
    assert np.isfinite(ones) and smoe.smoe_last_device_status() == smoe.SMOE_OK
