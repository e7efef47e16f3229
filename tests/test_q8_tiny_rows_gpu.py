"""Rows of the smallest numbers: 127 / top is beyond f32 below 3.8e-37, and the
codes are those of the values all the same.

Tolerance: half a step, and for the quotient, its product with the value and the
activation's own roundings (u = 2^-24) 127 steps times 26 u, as at other sizes;
a value of the activation below 2^-126 is off by 2^-149 or two of them besides."""
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


def _quantize(smoe, x, dt, act, cols):
    n = x.shape[0]
    q = torch.full((n, cols), 99, dtype=torch.int8, device="cuda")
    s = torch.full((n,), -7.0, device="cuda")
    smoe.smoe_quantize_rows_q8(x, DT[dt][0], act, n, cols, q, s)
    assert smoe.smoe_last_device_status() == smoe.SMOE_OK
    return q.cpu().numpy().astype(np.float64), s.cpu().numpy()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(30, 64), (30, 65), (700, 64), (700, 33), (30, 9000)])
@pytest.mark.parametrize("act", [0, 1])
def test_codes_of_tiny_rows(smoe, dt, rows, cols, act):
    g = torch.Generator().manual_seed(cols)
    # largest values from 1e-39 (below the normal numbers) over the border at 3.8e-37 to 1e-35
    v = torch.rand(rows, cols, generator=g, dtype=torch.float64) * 2 - 1
    v = v / v.abs().amax(1, keepdim=True) * torch.logspace(-39, -35, rows, dtype=torch.float64)[:, None]
    v[:, 1] = 0
    v = v.to(DT[dt][1])
    if act:  # SiLU(3) = 2.857..
        x = torch.cat([torch.full_like(v, 3.0), v], 1)
        want = v.double().numpy() * 3 / (1 + np.exp(-3.0))
    else:
        x, want = v, v.double().numpy()
    q, s = _quantize(smoe, x.cuda(), dt, act, cols)
    top = np.abs(want).max(1)
    least = 2.0 ** -148 if act else 0.0
    if act:
        assert (np.abs(s - top / 127) <= 12 * U * top / 127 + 2.0 ** -149).all()
    else:
        np.testing.assert_array_equal(s, top.astype(np.float32) / np.float32(127))
    step = (top / 127)[:, None]
    assert (np.abs(q * step - want) <= (0.5 + 127 * 26 * U) * step + least).all()
    assert (q[:, 1] == 0).all() and (np.abs(q).max(1) == 127).all()


@pytest.mark.parametrize("rows", [2, 700])
def test_the_smallest_number_of_all(smoe, rows):
    x = torch.zeros(rows, 32)
    x[:, 3], x[:, 4], x[:, 5] = 2.0 ** -149, -(2.0 ** -149), 2.0 ** -148
    x[0, 5] = 0
    q, _ = _quantize(smoe, x.cuda(), "f32", 0, 32)
    want = np.zeros((rows, 32))
    want[:, 3], want[:, 4], want[:, 5] = 64, -64, 127  # 63.5 to even
    want[0, 3], want[0, 4], want[0, 5] = 127, -127, 0
    np.testing.assert_array_equal(q, want)
