"""SiLU of large gates in the row quantiser: where e^-v is beyond the largest
numbers that a reciprocal can take, SiLU(v) is still a number, and up may
make it the largest of its row.

Tolerance (u = 2^-24): exp and the division are off by two units in the last
place each, the sum, two products and the scale by one rounding: 12 u; and e^v
below the smallest normal number is off by half of 2^-149 besides."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def smoe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build_library()
    import moe_expert_ffn_smoe_gb300 as m
    return m


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [8, 15])
def test_silu_of_large_gates(smoe, dt, cols):
    gates = [-60.0, -80.0, -87.0, -87.5, -88.0, -88.5, -89.0, -90.0, 60.0, 87.5, 88.5, 90.0, 1e30]
    tt = {"f32": torch.float32, "bf16": torch.bfloat16}[dt]
    x = torch.zeros(len(gates), 2 * cols)
    x[:, 1] = torch.tensor(gates)
    x[:, cols + 1] = torch.tensor([2.0 ** 120 if v < 0 else 1.0 for v in gates])
    x = x.to(tt)
    silu = lambda v: v / (1 + math.exp(-v)) if v > -700 else 0.0  # noqa: E731
    want = np.zeros((len(gates), cols))
    for r in range(len(gates)):
        for c in range(cols):
            want[r, c] = silu(float(x[r, c])) * float(x[r, cols + c])
    q = torch.empty(len(gates), cols, dtype=torch.int8, device="cuda")
    s = torch.empty(len(gates), device="cuda")
    smoe.smoe_quantize_rows_q8(x.cuda(), smoe.SMOE_F32 if dt == "f32" else smoe.SMOE_BF16, smoe.SMOE_Q8_SILU_MUL, len(gates),
                               cols, q, s)
    assert smoe.smoe_last_device_status() == smoe.SMOE_OK
    top = np.abs(want).max(1)
    low = np.array([2.0 ** -150 / math.exp(v) if v < -87 else 0.0 for v in x[:, 1].double().tolist()])
    got = s.double().cpu().numpy()
    assert (np.abs(got - top / 127) <= (12 * U + low) * top / 127).all(), (got * 127, top)
    codes = q.cpu().numpy()
    assert (codes[:, 1] == np.where(want[:, 1] > 0, 127, -127)).all()
    assert (np.delete(codes, 1, 1) == 0).all()


def test_silu_of_infinite_gates_is_no_number(smoe):
    """inf / (1 + e^inf) has no value: the row is one that is not finite."""
    x = torch.ones(3, 32, device="cuda")
    x[0, 3], x[1, 3], x[2, 3] = float("-inf"), float("inf"), float("nan")
    q = torch.full((3, 16), 9, dtype=torch.int8, device="cuda")
    s = torch.empty(3, device="cuda")
    smoe.smoe_quantize_rows_q8(x, smoe.SMOE_F32, smoe.SMOE_Q8_SILU_MUL, 3, 16, q, s)
    assert torch.isnan(s).all() and (q == 0).all()
