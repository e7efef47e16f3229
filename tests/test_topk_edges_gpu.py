"""Selections of NaN among masked logits, in every form that a row's length and
k choose: a NaN ranks below -inf, so it is selected once the -infs are fewer
than k, and it then has its index and the weight NaN wherever it stands."""
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


@pytest.mark.parametrize("E", [4, 8, 40, 100, 200, 500, 600, 1024, 2100])
@pytest.mark.parametrize("k", [1, 3, 4, 16, 17, 40])
@pytest.mark.parametrize("T", [1, 1100])
def test_topk_of_masked_and_nan(smoe, E, k, T):
    """Rows of -inf and NaN alone: k - 1, k and k + 1 masked (as far as the
    row goes), the NaNs before, behind and among them, none masked, all."""
    if k > E:
        pytest.skip("k > n_experts")
    rows, ref = [], []
    for masked in sorted({0, 1, k - 1, k, k + 1, E} & set(range(E + 1))):
        for where in ("behind", "before", "among"):
            at = {"behind": range(masked), "before": range(E - masked, E),
                  "among": sorted((7 * i) % E for i in range(masked)) if E % 7 else range(masked)}[where]
            row = torch.full((E,), float("nan"))
            row[list(at)] = float("-inf")
            nans = torch.isnan(row).nonzero().flatten().tolist()
            took = min(masked, k)
            rows.append(row)
            ref.append([-1] * took + nans[:k - took])
    n = len(rows)
    l = torch.stack([rows[t % n] for t in range(max(T, n))]).cuda()
    T = l.shape[0]
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), -7.0, device="cuda")
    smoe.smoe_topk_rows(l, T, E, E, k, idx, w)
    assert smoe.smoe_last_device_status() == smoe.SMOE_OK
    want = torch.tensor([ref[t % n] for t in range(T)], dtype=torch.int32, device="cuda")
    assert torch.equal(idx, want)
    assert torch.equal(torch.isnan(w), want >= 0)
    assert (w[want < 0] == 0).all()
