"""Refusals of the routing by scores, and the plain form that the GPU's is held to."""
import numpy as np
import pytest

import f8_util as u

A = 1 << 20
MB = 1 << 20


@pytest.fixture(scope="module")
def smoe():
    import __graft_entry__
    __graft_entry__.build_library()
    import moe_expert_ffn_smoe_gb300 as m
    return m


def test_route_rows_refusals(smoe):
    L = smoe._lib

    def f(lg=A, T=16, n=128, ld=128, b=A + MB, sc=1, G=8, tg=4, best=2, k=8, norm=1, scale=1.0, ix=A + 2 * MB, w=A + 3 * MB):
        return L.smoe_route_rows(lg, T, n, ld, b, sc, G, tg, best, k, norm, scale, ix, w, None)

    for bad in (dict(T=-1), dict(n=0), dict(n=1032, ld=1032), dict(k=0), dict(k=65), dict(n=4, ld=4, G=1, tg=1), dict(ld=127),
                dict(sc=2), dict(sc=-1), dict(G=0), dict(G=3), dict(n=1024, ld=1024, G=64), dict(tg=0), dict(tg=9), dict(best=0),
                dict(best=3), dict(G=64, tg=1), dict(G=16, tg=1, k=9), dict(scale=0.0), dict(scale=float("inf")),
                dict(scale=float("nan")), dict(T=(1 << 30) // 8 + 1)):
        assert f(**bad) == smoe.SMOE_ERR_SHAPE, bad
    for bad in (dict(lg=None), dict(ix=None), dict(w=None)):
        assert f(**bad) == smoe.SMOE_ERR_NULL, bad
    for bad in (dict(lg=A + 2), dict(b=A + MB + 1), dict(ix=A + 2 * MB + 2), dict(w=A + 3 * MB + 1)):
        assert f(**bad) == smoe.SMOE_ERR_ALIGN, bad
    for bad in (dict(w=A + 2 * MB + 4), dict(ix=A + 16), dict(w=A + MB + 508), dict(ix=A + 15 * 200 * 4 + 508, ld=200)):
        assert f(**bad) == smoe.SMOE_ERR_ALIAS, bad
    assert f(T=0, lg=None, ix=None, w=None) == smoe.SMOE_OK


def test_route_rows_backward_refusals(smoe):
    L = smoe._lib

    def f(lg=A, T=16, n=128, ld=128, sc=1, k=8, norm=1, scale=1.0, ix=A + MB, w=A + 2 * MB, dw=A + 3 * MB, dl=A + 4 * MB):
        return L.smoe_route_rows_backward(lg, T, n, ld, sc, k, norm, scale, ix, w, dw, dl, None)

    for bad in (dict(T=-1), dict(n=0), dict(n=1025, ld=1025), dict(k=0), dict(k=129), dict(ld=100), dict(sc=2), dict(scale=0.0)):
        assert f(**bad) == smoe.SMOE_ERR_SHAPE, bad
    for bad in (dict(lg=None), dict(ix=None), dict(w=None), dict(dw=None), dict(dl=None)):
        assert f(**bad) == smoe.SMOE_ERR_NULL, bad
    for bad in (dict(dl=A + 4 * MB + 4), dict(dw=A + 3 * MB + 2)):
        assert f(**bad) == smoe.SMOE_ERR_ALIGN, bad
    for bad in (dict(dl=A + 16), dict(dl=A + 3 * MB)):
        assert f(**bad) == smoe.SMOE_ERR_ALIAS, bad
    assert f(T=0, lg=None) == smoe.SMOE_OK


def test_binding_converts_floats(smoe):
    ok = (A, 0, 128, 128, None, 1, 8, 4, 2, 8, 1)
    smoe.smoe_route_rows(*ok, 2.5, A, A, stream=0)  # no tokens: nothing is launched
    smoe.smoe_route_rows(*ok, 1, A, A, stream=0)
    with pytest.raises(TypeError):
        smoe.smoe_route_rows(*ok, "1", A, A, stream=0)
    with pytest.raises(smoe.SmoeError) as ei:
        smoe.smoe_route_rows(*ok, 0.0, A, A, stream=0)
    assert ei.value.status == smoe.SMOE_ERR_SHAPE
    for name in ("smoe_route_rows", "smoe_route_rows_backward", "smoe_quantize_rows_f8", "smoe_quantize_blocks_f8",
                 "smoe_matmul_f8", "smoe_experts_matmul_f8", "smoe_experts_weight_grad"):
        assert callable(getattr(smoe._binding_f8, name)) and callable(smoe._by_ctypes(name))
    args = (A, 16, 128, 64, None, 1, 8, 4, 2, 8, 1, 1.0, A + MB, A + 2 * MB, 0)
    assert smoe._binding_f8.smoe_route_rows(*args) == smoe._by_ctypes("smoe_route_rows")(*args) == smoe.SMOE_ERR_SHAPE


@pytest.mark.parametrize("softmax", [True, False])
@pytest.mark.parametrize("norm", [True, False])
def test_the_gradient_is_that_of_differences(softmax, norm):
    """The formula that the GPU's gradient is held to, against central differences
    of the weights in float64 (error: h^2 / 6 of a third derivative, and 2^-53 / h)."""
    rng = np.random.default_rng(3)
    T, n, k, scale, h = 5, 12, 4, 2.5, 1e-5
    l = rng.normal(size=(T, n))
    l[1, :3] = -np.inf
    idx = u.choose(l, None, softmax, 1, 1, 1, k)
    idx[2, 1] = -1
    dw = rng.normal(size=(T, k))
    d, mag = u.weights_gradient(l, idx, softmax, norm, scale, dw)
    for t in range(T):
        for j in range(n):
            if l[t, j] == -np.inf:
                assert d[t, j] == 0
                continue
            v = []
            for s in (h, -h):
                x = l.copy()
                x[t, j] += s
                v.append((u.weights(x, idx, softmax, norm, scale)[t] * dw[t]).sum())
            assert abs((v[0] - v[1]) / (2 * h) - d[t, j]) <= 1e-9 * (1 + np.abs(mag[t]).sum())


def test_codes_of_the_plain_quantiser():
    v = u.e4m3(np.arange(256))
    assert v[0x7e] == 448 and v[0x08] == 2.0 ** -6 and v[1] == 2.0 ** -9 and np.isnan(v[[0x7f, 0xff]]).all()
    fine = np.array([c for c in range(256) if c & 0x7f != 0x7f])
    assert (u.to_e4m3(v[fine]) == fine).all()
    assert u.to_e4m3(np.array([17.0])) == u.to_e4m3(np.array([16.0])) and u.to_e4m3(np.array([19.0])) == u.to_e4m3(np.array([20.0]))
