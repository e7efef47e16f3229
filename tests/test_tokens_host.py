"""Refusals of the many-token and 8-bit calls, which check every argument on
the host before any launch (the addresses below are never dereferenced)."""
import ctypes

import pytest

A = 1 << 20
MB = 1 << 20
BAD = ctypes.c_size_t(-1).value


@pytest.fixture(scope="module")
def smoe():
    import __graft_entry__
    __graft_entry__.build_library()
    import moe_expert_ffn_smoe_gb300 as m
    return m


def test_topk_rows_refusals(smoe):
    L = smoe._lib

    def f(lg=A, T=16, E=128, ld=128, k=8, ix=A + MB, w=A + 2 * MB):
        return L.smoe_topk_rows(lg, T, E, ld, k, ix, w, None)

    for bad in (dict(T=-1), dict(E=0), dict(E=smoe.SMOE_MAX_ROUTE_EXPERTS + 1, ld=10000), dict(k=0), dict(k=129),
                dict(k=smoe.SMOE_MAX_TOP_K + 1), dict(ld=127), dict(T=(1 << 30) // 8 + 1)):
        assert f(**bad) == smoe.SMOE_ERR_SHAPE, bad
    for bad in (dict(lg=None), dict(ix=None), dict(w=None)):
        assert f(**bad) == smoe.SMOE_ERR_NULL, bad
    for bad in (dict(lg=A + 2), dict(ix=A + MB + 1), dict(w=A + 2 * MB + 2)):
        assert f(**bad) == smoe.SMOE_ERR_ALIGN, bad
    assert f(w=A + MB + 4) == smoe.SMOE_ERR_ALIAS
    assert f(ix=A + 15 * 200 * 4 + 508, ld=200) == smoe.SMOE_ERR_ALIAS  # the last row's end, by the pitch
    assert f(T=0, lg=None, ix=None, w=None) == smoe.SMOE_OK

    def g(ix=A, w=A + MB, dw=A + 2 * MB, T=16, E=128, k=8, dl=A + 3 * MB):
        return L.smoe_topk_rows_backward(ix, w, dw, T, E, k, dl, None)

    for bad in (dict(T=-1), dict(E=0), dict(k=0), dict(E=4)):
        assert g(**bad) == smoe.SMOE_ERR_SHAPE, bad
    for bad in (dict(ix=None), dict(w=None), dict(dw=None), dict(dl=None)):
        assert g(**bad) == smoe.SMOE_ERR_NULL, bad
    assert g(dl=A + 3 * MB + 8) == smoe.SMOE_ERR_ALIGN
    assert g(dl=A + 16) == smoe.SMOE_ERR_ALIAS
    assert g(T=0, ix=None) == smoe.SMOE_OK


def test_dispatch_refusals(smoe):
    L = smoe._lib
    need = L.smoe_dispatch_workspace_bytes(16, 8, 128)
    assert 0 < need < MB and need % 256 == 0
    assert L.smoe_dispatch_workspace_bytes(0, 8, 128) == 0
    for bad in ((-1, 8, 128), (16, 0, 128), (16, 65, 128), (16, 8, 0), (16, 8, smoe.SMOE_MAX_ROUTE_EXPERTS + 1)):
        assert L.smoe_dispatch_workspace_bytes(*bad) == BAD

    def f(ix=A, T=16, k=8, E=128, x=A + MB, dt=0, d=64, of=A + 2 * MB, o=A + 3 * MB, p=A + 4 * MB, xs=A + 5 * MB,
          ws=A + 6 * MB, n=need):
        return L.smoe_dispatch_tokens(ix, T, k, E, x, dt, d, of, o, p, xs, ws, n, None)

    for bad in (dict(T=-1), dict(k=0), dict(E=0), dict(E=9000), dict(dt=2), dict(dt=-1), dict(d=-1)):
        assert f(**bad) == smoe.SMOE_ERR_SHAPE, bad
    for bad in (dict(ix=None), dict(of=None), dict(o=None), dict(p=None), dict(x=None), dict(xs=None)):
        assert f(**bad) == smoe.SMOE_ERR_NULL, bad
    for bad in (dict(ix=A + 2), dict(of=A + 2 * MB + 1), dict(o=A + 3 * MB + 2), dict(p=A + 4 * MB + 2),
                dict(x=A + MB + 2), dict(xs=A + 5 * MB + 1), dict(ws=A + 6 * MB + 8), dict(dt=1, x=A + MB + 1)):
        assert f(**bad) == smoe.SMOE_ERR_ALIGN, bad
    for bad in (dict(ws=None), dict(n=need - 1)):
        assert f(**bad) == smoe.SMOE_ERR_WORKSPACE, bad
    for bad in (dict(p=A + 3 * MB + 4), dict(xs=A + MB + 64), dict(o=A + 16), dict(ws=A + 5 * MB + 16 * 8 * 64 * 4 - 16),
                dict(of=A + 6 * MB)):
        assert f(**bad) == smoe.SMOE_ERR_ALIAS, bad


def test_combine_and_gradients_refusals(smoe):
    L = smoe._lib

    def c(ys=A, dt=0, p=A + MB, w=A + 2 * MB, T=16, k=8, d=64, out=A + 3 * MB):
        return L.smoe_combine_tokens(ys, dt, p, w, T, k, d, out, None)

    def b(ys=A, dt=0, p=A + MB, T=16, k=8, d=64, out=A + 3 * MB):
        return L.smoe_dispatch_tokens_backward(ys, dt, p, T, k, d, out, None)

    for f in (c, b):
        for bad in (dict(T=-1), dict(k=0), dict(k=65), dict(dt=3), dict(d=-1), dict(d=(1 << 30) + 1)):
            assert f(**bad) == smoe.SMOE_ERR_SHAPE, bad
        for bad in (dict(ys=None), dict(p=None), dict(out=None)):
            assert f(**bad) == smoe.SMOE_ERR_NULL, bad
        assert f(out=A + 16) == smoe.SMOE_ERR_ALIAS
        assert f(out=A + 3 * MB + 2) == smoe.SMOE_ERR_ALIGN
        assert f(T=0, ys=None) == smoe.SMOE_OK
        assert f(d=0, ys=None) == smoe.SMOE_OK
    assert c(w=None) == smoe.SMOE_ERR_NULL

    def g(do=A, ys=A + MB, dt=0, p=A + 2 * MB, w=A + 3 * MB, T=16, k=8, d=64, dy=A + 4 * MB, dw=A + 5 * MB):
        return L.smoe_combine_tokens_backward(do, ys, dt, p, w, T, k, d, dy, dw, None)

    for bad in (dict(T=-1), dict(k=0), dict(dt=2), dict(d=-4)):
        assert g(**bad) == smoe.SMOE_ERR_SHAPE, bad
    for bad in (dict(do=None), dict(ys=None), dict(p=None), dict(w=None), dict(dy=None), dict(dw=None)):
        assert g(**bad) == smoe.SMOE_ERR_NULL, bad
    for bad in (dict(dy=A + MB + 256), dict(dw=A + 4 * MB + 4), dict(dw=A + 3 * MB)):
        assert g(**bad) == smoe.SMOE_ERR_ALIAS, bad
    assert g(T=0) == smoe.SMOE_OK


def test_q8_refusals(smoe):
    L = smoe._lib

    def q(x=A, dt=0, act=0, r=16, c=64, q=A + MB, s=A + 2 * MB):
        return L.smoe_quantize_rows_q8(x, dt, act, r, c, q, s, None)

    for bad in (dict(r=-1), dict(c=-1), dict(c=smoe.SMOE_MAX_COLS + 1), dict(dt=2), dict(act=2)):
        assert q(**bad) == smoe.SMOE_ERR_SHAPE, bad
    for bad in (dict(x=None), dict(q=None), dict(s=None)):
        assert q(**bad) == smoe.SMOE_ERR_NULL, bad
    for bad in (dict(x=A + 2), dict(q=A + MB + 8), dict(s=A + 2 * MB + 2)):
        assert q(**bad) == smoe.SMOE_ERR_ALIGN, bad
    assert q(q=A + 16 * 64 * 4 - 16) == smoe.SMOE_ERR_ALIAS
    assert q(act=1, q=A + 16 * 64 * 8 - 16) == smoe.SMOE_ERR_ALIAS  # rows of 2 cols
    assert q(r=0, x=None) == smoe.SMOE_OK

    need = L.smoe_experts_matmul_q8_workspace_bytes(16, 128, 8, 96, 256)
    assert 0 < need < MB
    assert L.smoe_matmul_q8_workspace_bytes(0, 96, 256) == 0
    for bad in ((16, 128, 8, 96, 250), (16, -1, 8, 96, 256), (16, 128, 0, 96, 256), (16, 128, 8, -1, 256),
                (16, 128, 8, 96, 32784)):
        assert L.smoe_experts_matmul_q8_workspace_bytes(*bad) == BAD

    def m(xq=A, xs=A + MB, ns=16, o=A + 2 * MB, k=8, of=A + 3 * MB, r=128, E=8, wq=A + 4 * MB, s=A + 5 * MB, N=96,
          K=256, y=A + 6 * MB, dt=1, ws=A + 7 * MB, n=need):
        return L.smoe_experts_matmul_q8(xq, xs, ns, o, k, of, r, E, wq, s, N, K, y, dt, ws, n, None)

    for bad in (dict(K=250), dict(K=-16), dict(r=-1), dict(E=0), dict(N=-1), dict(dt=5), dict(k=0), dict(o=None),
                dict(E=8192, N=1 << 18)):
        assert m(**bad) == smoe.SMOE_ERR_SHAPE, bad  # o None: 128 rows of an xq of 16
    for bad in (dict(xq=None), dict(xs=None), dict(of=None), dict(wq=None), dict(s=None), dict(y=None)):
        assert m(**bad) == smoe.SMOE_ERR_NULL, bad
    for bad in (dict(xq=A + 8), dict(wq=A + 4 * MB + 4), dict(s=A + 5 * MB + 4), dict(y=A + 6 * MB + 2),
                dict(ws=A + 7 * MB + 4), dict(o=A + 2 * MB + 2)):
        assert m(**bad) == smoe.SMOE_ERR_ALIGN, bad
    for bad in (dict(ws=None), dict(n=need - 1)):
        assert m(**bad) == smoe.SMOE_ERR_WORKSPACE, bad
    for bad in (dict(y=A + 4 * MB + 64), dict(ws=A + 6 * MB), dict(y=A + 16)):
        assert m(**bad) == smoe.SMOE_ERR_ALIAS, bad
    assert m(r=0, xq=None) == smoe.SMOE_OK
    assert m(N=0, xq=None) == smoe.SMOE_OK
    assert L.smoe_matmul_q8(A, A + MB, 16, A + 2 * MB, A + 3 * MB, 96, 250, A + 4 * MB, 0, A + 5 * MB, MB, None) == \
        smoe.SMOE_ERR_SHAPE


def test_binding_converts_and_refuses(smoe):
    """Addresses, None and objects with data_ptr(); sizes beyond 32 bits and
    other objects are refused before the library is called."""
    class Buf:
        def data_ptr(self):
            return A

    ok = (Buf(), 0, 128, 128, 8, None, A)
    smoe.smoe_topk_rows(*ok, stream=0)  # no tokens: nothing is launched
    with pytest.raises(smoe.SmoeError) as ei:
        smoe.smoe_topk_rows(A, 16, 128, 64, 8, A + MB, A + 2 * MB, stream=0)
    assert ei.value.status == smoe.SMOE_ERR_SHAPE
    with pytest.raises(OverflowError):
        smoe.smoe_topk_rows(A, 1 << 40, 128, 128, 8, A, A, stream=0)
    with pytest.raises(AttributeError):
        smoe.smoe_topk_rows("x", 0, 128, 128, 8, A, A, stream=0)
    with pytest.raises(TypeError):
        smoe.smoe_topk_rows(A, 1.5, 128, 128, 8, A, A, stream=0)
    with pytest.raises(TypeError):
        smoe._binding.smoe_topk_rows(A, 0)
    # the two routes to the library agree on every refusal
    for args in ((A, -1, 128, 128, 8, A, A, 0), (None, 16, 128, 128, 8, A, A, 0), (A + 2, 16, 128, 128, 8, A + MB, A + 2 * MB, 0),
                 (A, 16, 128, 128, 8, A + MB, A + MB, 0)):
        assert smoe._binding.smoe_topk_rows(*args) == smoe._lib.smoe_topk_rows(*args) != 0
