"""Refusals of the 8-bit floating-point calls and of the weights' gradient (the
addresses below are never dereferenced)."""
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


def test_quantisers_refusals(smoe):
    L = smoe._lib

    def q(x=A, dt=0, act=0, r=16, c=300, q=A + MB, s=A + 2 * MB):
        return L.smoe_quantize_rows_f8(x, dt, act, r, c, q, s, None)

    for bad in (dict(r=-1), dict(c=-1), dict(c=smoe.SMOE_MAX_COLS + 1), dict(dt=2), dict(act=2), dict(r=(1 << 30) + 1)):
        assert q(**bad) == smoe.SMOE_ERR_SHAPE, bad
    for bad in (dict(x=None), dict(q=None), dict(s=None)):
        assert q(**bad) == smoe.SMOE_ERR_NULL, bad
    for bad in (dict(x=A + 2), dict(q=A + MB + 8), dict(s=A + 2 * MB + 2)):
        assert q(**bad) == smoe.SMOE_ERR_ALIGN, bad
    assert q(q=A + 16 * 300 * 4 - 16) == smoe.SMOE_ERR_ALIAS
    assert q(act=1, q=A + 16 * 300 * 8 - 16) == smoe.SMOE_ERR_ALIAS  # rows of 2 cols
    assert q(s=A + MB + 16 * 300 - 4) == smoe.SMOE_ERR_ALIAS
    assert q(q=A + 2 * MB + 16 * 3 * 4 - 16) == smoe.SMOE_ERR_ALIAS  # three scales a row
    assert q(r=0, x=None) == smoe.SMOE_OK and q(c=0, x=None) == smoe.SMOE_OK

    def b(w=A, dt=1, n=2, r=130, c=200, q=A + MB, s=A + 2 * MB, qt=A + 3 * MB, st=A + 4 * MB):
        return L.smoe_quantize_blocks_f8(w, dt, n, r, c, q, s, qt, st, None)

    for bad in (dict(n=-1), dict(r=-1), dict(c=-1), dict(dt=3), dict(n=1 << 20, r=1 << 11), dict(n=1 << 20, c=1 << 11),
                dict(n=1, r=1 << 30, c=1 << 20)):
        assert b(**bad) == smoe.SMOE_ERR_SHAPE, bad
    for bad in (dict(w=None), dict(q=None), dict(s=None), dict(qt=None), dict(st=None)):
        assert b(**bad) == smoe.SMOE_ERR_NULL, bad
    for bad in (dict(w=A + 1), dict(q=A + MB + 4), dict(qt=A + 3 * MB + 8), dict(s=A + 2 * MB + 2), dict(st=A + 4 * MB + 1)):
        assert b(**bad) == smoe.SMOE_ERR_ALIGN, bad
    for bad in (dict(qt=A + MB + 2 * 130 * 200 - 16), dict(q=A + 2 * 130 * 200 * 2 - 16), dict(st=A + 2 * MB + 28)):
        assert b(**bad) == smoe.SMOE_ERR_ALIAS, bad
    assert b(n=0, w=None) == smoe.SMOE_OK and b(r=0, w=None) == smoe.SMOE_OK


def test_product_refusals(smoe):
    L = smoe._lib
    need = L.smoe_experts_matmul_f8_workspace_bytes(16, 128, 8, 96, 256)
    assert 0 < need < MB
    assert L.smoe_matmul_f8_workspace_bytes(0, 96, 256) == 0
    for bad in ((16, 128, 8, 96, 250), (16, -1, 8, 96, 256), (16, 128, 0, 96, 256), (16, 128, 8, -1, 256), (16, 128, 8, 96, 32784),
                (0, 128, 8, 96, 256)):
        assert L.smoe_experts_matmul_f8_workspace_bytes(*bad) == BAD
    sizes = [L.smoe_experts_matmul_f8_workspace_bytes(r, r, 8, 96, 256) for r in range(1, 3000, 7)]
    assert sizes == sorted(sizes)

    def m(xq=A, xs=A + MB, ns=16, o=A + 2 * MB, k=8, of=A + 3 * MB, r=128, E=8, wq=A + 4 * MB, s=A + 5 * MB, N=96,
          K=256, y=A + 6 * MB, dt=1, ws=A + 7 * MB, n=need):
        return L.smoe_experts_matmul_f8(xq, xs, ns, o, k, of, r, E, wq, s, N, K, y, dt, ws, n, None)

    for bad in (dict(K=250), dict(K=-16), dict(r=-1), dict(E=0), dict(N=-1), dict(dt=5), dict(k=0), dict(k=65), dict(o=None),
                dict(E=8192, N=1 << 18), dict(ns=0)):
        assert m(**bad) == smoe.SMOE_ERR_SHAPE, bad  # o None: 128 rows of an xq of 16
    for bad in (dict(xq=None), dict(xs=None), dict(of=None), dict(wq=None), dict(s=None), dict(y=None)):
        assert m(**bad) == smoe.SMOE_ERR_NULL, bad
    for bad in (dict(xq=A + 8), dict(wq=A + 4 * MB + 4), dict(s=A + 5 * MB + 2), dict(y=A + 6 * MB + 2),
                dict(ws=A + 7 * MB + 4), dict(o=A + 2 * MB + 2), dict(of=A + 3 * MB + 1), dict(xs=A + MB + 2)):
        assert m(**bad) == smoe.SMOE_ERR_ALIGN, bad
    for bad in (dict(ws=None), dict(n=need - 1)):
        assert m(**bad) == smoe.SMOE_ERR_WORKSPACE, bad
    for bad in (dict(y=A + 4 * MB + 64), dict(ws=A + 6 * MB), dict(y=A + 16), dict(y=A + MB + 16 * 2 * 4 - 16),
                dict(y=A + 5 * MB + 8 * 2 * 4 - 16)):
        assert m(**bad) == smoe.SMOE_ERR_ALIAS, bad
    assert m(r=0, xq=None) == smoe.SMOE_OK and m(N=0, xq=None) == smoe.SMOE_OK
    assert L.smoe_matmul_f8(A, A + MB, 16, A + 2 * MB, A + 3 * MB, 96, 250, A + 4 * MB, 0, A + 5 * MB, MB, None) == \
        smoe.SMOE_ERR_SHAPE


def test_weight_grad_refusals(smoe):
    L = smoe._lib

    def g(dy=A, x=A + MB, of=A + 2 * MB, r=64, E=4, N=96, K=256, acc=0, dw=A + 3 * MB, dt=0):
        return L.smoe_experts_weight_grad(dy, x, of, r, E, N, K, acc, dw, dt, None)

    for bad in (dict(r=-1), dict(r=(1 << 30) + 1), dict(E=0), dict(E=8193), dict(N=-8), dict(N=100), dict(K=4), dict(K=-8),
                dict(N=smoe.SMOE_MAX_COLS + 8), dict(K=smoe.SMOE_MAX_COLS + 8), dict(dt=2)):
        assert g(**bad) == smoe.SMOE_ERR_SHAPE, bad
    for bad in (dict(dy=None), dict(x=None), dict(of=None), dict(dw=None)):
        assert g(**bad) == smoe.SMOE_ERR_NULL, bad
    for bad in (dict(dy=A + 8), dict(x=A + MB + 2), dict(of=A + 2 * MB + 2), dict(dw=A + 3 * MB + 8)):
        assert g(**bad) == smoe.SMOE_ERR_ALIGN, bad
    for bad in (dict(dw=A + 16), dict(dw=A + MB + 64 * 256 * 2 - 16), dict(dw=A + 2 * MB + 16)):
        assert g(**bad) == smoe.SMOE_ERR_ALIAS, bad
    assert g(N=0, dy=None) == smoe.SMOE_OK and g(K=0, dy=None) == smoe.SMOE_OK
    assert g(r=0, acc=1, dy=None, x=None, dw=None) == smoe.SMOE_OK  # nothing to add
