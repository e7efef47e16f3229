"""The row quantiser's forms for many rows (two and four warps a row, from four
rows an SM on), code by code: at, below and above the lengths up to which a form
keeps a row between its two passes, in vectors and in single elements."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f32": (0, torch.float32), "bf16": (1, torch.bfloat16)}


@pytest.fixture(scope="module")
def smoe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build_library()
    import moe_expert_ffn_smoe_gb300 as m
    return m


@pytest.fixture(scope="module")
def rows():
    return 4 * torch.cuda.get_device_properties(0).multi_processor_count


def _quantize(smoe, x, dt, act, cols):
    n = x.shape[0]
    buf = torch.full((n * cols + 64,), 99, dtype=torch.int8, device="cuda")
    s = torch.full((n + 16,), -7.0, device="cuda")
    smoe.smoe_quantize_rows_q8(x, DT[dt][0], act, n, cols, buf, s)
    assert smoe.smoe_last_device_status() == smoe.SMOE_OK
    assert (buf[n * cols:] == 99).all() and (s[n:] == -7).all()
    return buf[:n * cols].view(n, cols).cpu().numpy(), s[:n].cpu().numpy()


# f32 and bf16 rows in vectors up to 4096 and 8192 columns, single elements up to 512 and 1024
@pytest.mark.parametrize("dt,cols", [(d, c) for d in ("f32", "bf16") for c in (8, 512, 4096, 4104, 8192, 8200, 511, 513, 1023, 1025)])
@pytest.mark.parametrize("more", [-1, 0, 3])
def test_plain_rows(smoe, rows, dt, cols, more):
    n = rows + more
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = (torch.randn(n, cols, generator=g, device="cuda") * torch.logspace(-6, 6, n, device="cuda")[:, None]).to(DT[dt][1])
    x[1] = 0
    x[2, -1] = float("nan")
    x[n - 1, 0] = float("-inf")
    # ties: the scale's reciprocal is exactly 1 and every other value halfway between two codes
    x[3] = ((torch.arange(cols, device="cuda") * 2) % 254 - 127).float() / 2
    x[3, 0] = 127.0
    q, s = _quantize(smoe, x, dt, smoe.SMOE_Q8_PLAIN, cols)
    v = x.float().cpu().numpy()
    bad = ~np.isfinite(v).all(1)
    v[bad] = 0
    top = np.abs(v).max(1, keepdims=True)
    up = np.where(top > 0, np.float32(127) / np.where(top > 0, top, 1), np.float32(0)).astype(np.float32)
    np.testing.assert_array_equal(q, np.rint((v * up).astype(np.float32)).astype(np.int8))
    np.testing.assert_array_equal(s, np.where(bad, np.float32("nan"), (top / np.float32(127))[:, 0]))
    assert bad.tolist() == [r in (2, n - 1) for r in range(n)]


# half as many columns as the plain rows
@pytest.mark.parametrize("dt,cols", [(d, c) for d in ("f32", "bf16") for c in (8, 2048, 2056, 4096, 4104, 511, 513, 1023, 1025)])
@pytest.mark.parametrize("more", [-1, 3])
def test_rows_of_the_activation(smoe, rows, dt, cols, more):
    n = rows + more
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = (3 * torch.randn(n, 2 * cols, generator=g, device="cuda")).to(DT[dt][1])
    x[1, cols:] = 0
    q, s = _quantize(smoe, x, dt, smoe.SMOE_Q8_SILU_MUL, cols)
    v = x.double().cpu().numpy()
    ga, up = v[:, :cols], v[:, cols:]
    ref = ga / (1 + np.exp(-ga)) * up
    top = np.abs(ref).max(1)
    # exp and the division (2 units in the last place each), the sum, two products, the scale: 12 roundings at most
    np.testing.assert_allclose(s, top / 127, rtol=12 * U)
    # half a step, and the roundings of a value of up to 127 steps and of the step
    assert (np.abs(q * (top / 127)[:, None] - ref) <= (0.5 + 127 * 26 * U) * (top / 127)[:, None]).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 300])
def test_ties_go_to_the_even_code(smoe, dt, n):
    x = torch.zeros(n, 256)
    x[:, 0] = 127
    x[:, 1:] = torch.arange(-127, 128).float() - 0.5
    x[:, 1] = 0
    q, s = _quantize(smoe, x.to(DT[dt][1]).cuda(), dt, smoe.SMOE_Q8_PLAIN, 256)
    assert (s == 1).all()
    np.testing.assert_array_equal(q, np.rint(x.numpy()).astype(np.int8))
