"""The codes after the activation are those of the f32 steps
g / (1 + e^-g) u, which torch takes one by one: scales and codes are theirs."""
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


def quantised(smoe, x, K):
    """(values of the codes, scales) of rows [gate | up]."""
    R = x.shape[0]
    q = torch.full((R, K), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((R, -(-K // 128)), -7.0, device="cuda")
    smoe.smoe_quantize_rows_f8(x, int(x.dtype == torch.bfloat16), smoe.SMOE_Q8_SILU_MUL, R, K, q, s)
    assert smoe.smoe_last_device_status() == smoe.SMOE_OK
    return q.view(torch.float8_e4m3fn).float(), s


def steps(v, K):
    """The same of f32 values v [R, K], one torch operation a step."""
    v = torch.nn.functional.pad(v, (0, -K % 128)).view(v.shape[0], -1, 128)
    top = v.abs().amax(2, keepdim=True)
    four = torch.full_like(top, 448.0)
    lift = torch.where((four / top).isinf() & (top > 0), 2.0 ** 64, 1.0)  # 448 / top is beyond f32
    q = (v * lift * torch.where(top > 0, four / (top * lift), 0.0)).clamp(-448, 448).to(torch.float8_e4m3fn).float()
    return q.view(v.shape[0], -1)[:, :K], (top / four)[:, :, 0]


def holds(smoe, x, K):
    """Equal, but for a quotient in 2^21 that is rounded to the other side: that moves a
    scale only where it is its block's largest, a code only where it lies within 2^-23 of
    a border (a step is 2^-4 of it at least)."""
    q, s = quantised(smoe, x, K)
    g, up = x[:, :K].float(), x[:, K:].float()
    rq, rs = steps(g / (1 + torch.exp(-g)) * up, K)
    moved = (s - rs).abs()
    assert (moved <= 2.0 ** -23 * rs).all()  # one unit in the last place at most
    assert (moved > 0).sum().item() <= 1 + s.numel() * 2.0 ** -20
    off = q != rq
    # one code up or down, where a scale has moved or never
    assert ((q - rq).abs() <= rq.abs() / 8 + 2.0 ** -9).all()
    assert off.sum().item() <= 1 + q.numel() * 2.0 ** -40 + 128 * (moved > 0).sum().item()


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,K", [(2049, 1536), (301, 1000), (129, 77), (64, 16), (1, 1)])
def test_rows_of_activations(smoe, dt, R, K):
    g = torch.Generator(device="cuda").manual_seed(R)
    x = torch.randn(R, 2 * K, generator=g, device="cuda") * torch.exp(torch.randn(R, 1, generator=g, device="cuda"))
    holds(smoe, x.to(dt), K)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_every_bf16_gate(smoe, dt):
    """All finite ones above -88 (where e^-g leaves f32), alone in their block: the scale is theirs."""
    g = torch.arange(65536, device="cuda").to(torch.int32).bitwise_and(0xffff)
    g = (g << 16).view(torch.float32)
    g = g[g.isfinite() & (g > -88)]
    # from 2^-100 on: below, a remainder would lie under f32's smallest number
    g = g[(g.abs() >= 2.0 ** -100) & (g.abs() <= 2.0 ** 100)]
    x = torch.zeros(g.numel(), 256, device="cuda")
    x[:, 5], x[:, 128 + 5] = g, 1.5
    holds(smoe, x.to(dt), 128)


def test_gates_far_below_zero(smoe):
    """Down to where e^-g leaves f32, in a row with others and in one of their own;
    infinities and NaN make their block NaN alone."""
    K = 256
    gates = torch.tensor([-63.9, -64.0, -64.1, -80.0, -87.0, -87.4, -87.9, -88.0, -88.5, -95.0, -1e4], device="cuda")
    x = torch.zeros(len(gates) + 3, 2 * K, device="cuda")
    x[:11, 3], x[:11, K + 3] = gates, 2.0 ** 60
    x[:11, 200], x[:11, K + 200] = 2.0, 3.0
    for r, v in ((11, -np.inf), (12, np.inf), (13, np.nan)):
        x[r, 130], x[r, K + 130] = v, 1.0
        x[r, 3], x[r, K + 3] = 1.0, 1.0
    q, s = quantised(smoe, x, K)
    v = x[:11].double()
    v = v[:, :K] * torch.sigmoid(v[:, :K]) * v[:, K:]
    top = torch.stack([v[:, :128].abs().amax(1), v[:, 128:].abs().amax(1)], 1)
    # expf to two units, a product or quotient, its product and the scale, one each: 2^-22 and
    # three 2^-24, four times that; e^g below the normal numbers by half of 2^-149, times |g| 2^60
    bound = 2.0 ** -20 * top + torch.where(top < 1e-3, 100 * 2.0 ** (60 - 150), 0.0)
    assert ((s[:11].double() * 448 - top).abs() <= bound).all()
    assert (q[11:, 128:] == 0).all() and s[11:, 1].isnan().all() and s[11:, 0].isfinite().all()
    one = torch.tensor(1.0).sigmoid().item()
    assert torch.allclose(s[11:, 0] * 448, torch.full((3,), one, device="cuda"), rtol=2.0 ** -20)
