"""Offsets that do not ascend: ranges that overlap, whose tiles add up to more
than 32 bits count.  Reported, with nothing written outside the arrays."""
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


# every second expert's range is all rows: 4096 times 2^20 tiles of eight rows
# (no columns: the dots), 4096 times some 700,000 of 192 (the tensor cores)
@pytest.mark.parametrize("R,K", [(1 << 23, 0), (1 << 27, 16), (1 << 12, 0), (1 << 12, 16)])
def test_tiles_of_overlapping_ranges(smoe, R, K):
    E, N = 8192, 1
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1::2] = R
    order = torch.zeros(R, dtype=torch.int32, device="cuda")
    x = torch.ones(1, 16, dtype=torch.int8, device="cuda")
    w = torch.ones(E, 16, dtype=torch.int8, device="cuda")
    one = torch.ones(E, device="cuda")
    pad = 1 << 20
    y = torch.full((R + pad,), -7.0, device="cuda")
    need = smoe.smoe_experts_matmul_q8_workspace_bytes(1, R, E, N, K)
    ws = torch.full((need + 2 * pad,), 201, dtype=torch.uint8, device="cuda")
    smoe.smoe_experts_matmul_q8(x, one, 1, order, 1, off, R, E, w, one, N, K, y, smoe.SMOE_F32, ws.data_ptr() + pad, need)
    assert smoe.smoe_last_device_status() == smoe.SMOE_ERR_ROUTE
    assert (y[R:] == -7).all() and (ws[:pad] == 201).all() and (ws[pad + need:] == 201).all()
    # the next call, with offsets that ascend, is whole
    off[1:] = R
    smoe.smoe_experts_matmul_q8(x, one, 1, order, 1, off, R, E, w, one, N, K, y, smoe.SMOE_F32, ws.data_ptr() + pad, need)
    assert smoe.smoe_last_device_status() == smoe.SMOE_OK
    assert (y[:R] == K).all()
