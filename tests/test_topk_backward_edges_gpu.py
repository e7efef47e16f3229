"""The gradient of a selection some of whose slots were given no expert after
the selection: by -1, or by an index past the last expert, as the dispatch
takes them."""
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


@pytest.mark.parametrize("T,E,k", [(5, 12, 4), (33, 128, 8), (3, 600, 40)])
@pytest.mark.parametrize("gone", ["-1", "n", "n + 5", "-9"])
def test_slots_without_an_expert_count_for_nothing(smoe, T, E, k, gone):
    g = torch.Generator(device="cuda").manual_seed(T)
    l = torch.randn(T, E, generator=g, device="cuda")
    idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, k, device="cuda")
    smoe.smoe_topk_rows(l, T, E, E, k, idx, w)
    dw = torch.randn(T, k, generator=g, device="cuda")
    off = torch.rand(T, k, generator=g, device="cuda") < 0.4
    idx[off] = {"-1": -1, "n": E, "n + 5": E + 5, "-9": -9}[gone]
    dw[off] = float("nan")  # not read into anything
    dl = torch.full((T, E), float("nan"), device="cuda")
    smoe.smoe_topk_rows_backward(idx, w, dw, T, E, k, dl)
    assert smoe.smoe_last_device_status() == smoe.SMOE_OK
    wd, gd = torch.where(off, 0.0, w.double()), torch.where(off, 0.0, dw.double())
    c = (wd * gd).sum(1, keepdim=True)
    ref = torch.zeros(T, E, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(ref)
    at = torch.where(off, 0, idx).long()
    ref.scatter_add_(1, at, torch.where(off, 0.0, wd * (gd - c)))
    mag.scatter_add_(1, at, torch.where(off, 0.0, wd * (gd.abs() + (wd * gd.abs()).sum(1, keepdim=True))))
    # two products and five shuffles in c, the difference and the product: 9 roundings
    assert ((dl.double() - ref).abs() <= 9 * U * mag).all()
