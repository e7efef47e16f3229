"""Routing by scores on the GPU against float64: the choice exactly, weights and
gradients within the rounding of their f32 steps."""
import numpy as np
import pytest

import f8_util as u

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch

    import moe_expert_ffn_smoe_gb300 as smoe
    return torch, smoe, torch.device("cuda:0")


def rtol(n):
    """Of a weight: the exponential's argument is rounded (2^-24 of up to 20) and
    its value to 2 units (2^-22); a lane adds n / 32 terms and five more follow, in
    the score and in the sum of the chosen; some five more roundings."""
    return (20 + n / 32 + 32) * 2.0 ** -24 * 2


def route(env, l, b, softmax, G, tg, best, k, norm, scale, ld=None):
    torch, smoe, dev = env
    T, n = l.shape
    ld = ld or n
    L = torch.full((T, ld), float("nan"), device=dev)
    L[:, :n] = torch.from_numpy(l)
    B = None if b is None else torch.from_numpy(b).to(dev)
    idx = torch.full((T, k), -7, dtype=torch.int32, device=dev)
    w = torch.full((T, k), 7.0, device=dev)
    smoe.smoe_route_rows(L, T, n, ld, B, smoe.SMOE_SCORE_SOFTMAX if softmax else smoe.SMOE_SCORE_SIGMOID, G, tg, best, k,
                         int(norm), scale, idx, w)
    return L, idx, w


def check(env, l, b, softmax, G, tg, best, k, norm, scale=1.0, ld=None, dw=None):
    torch, smoe, dev = env
    T, n = l.shape
    L, idx, w = route(env, l, b, softmax, G, tg, best, k, norm, scale, ld)
    gi, gw = idx.cpu().numpy(), w.cpu().numpy().astype(np.float64)
    ref = u.choose(l, b, softmax, G, tg, best, k)
    assert (gi == ref).all(), np.argwhere(gi != ref)[:5]
    rw = u.weights(l, ref, softmax, norm, scale)
    assert (np.abs(gw - rw) <= rtol(n) * np.abs(rw) + 1e-37).all()
    if dw is None:
        return
    dl = torch.full((T, n), float("nan"), device=dev)
    smoe.smoe_route_rows_backward(L, T, n, ld or n, smoe.SMOE_SCORE_SOFTMAX if softmax else smoe.SMOE_SCORE_SIGMOID, k,
                                  int(norm), scale, idx, w, torch.from_numpy(dw.astype(np.float32)).to(dev), dl)
    d, mag = u.weights_gradient(l, ref, softmax, norm, scale, dw.astype(np.float32).astype(np.float64))
    # the weights' own rounding, the sum over the slots, and as much again
    assert (np.abs(dl.cpu().numpy() - d) <= 4 * (rtol(n) + k * 2.0 ** -23) * mag + 1e-36).all()


def logits(rng, T, n, masked=True):
    l = rng.normal(size=(T, n)).astype(np.float32)
    if masked:
        l[rng.random((T, n)) < 0.1] = -np.inf
        l[rng.random(T) < 0.1] = -np.inf
    return l


@pytest.mark.parametrize("softmax", [True, False])
@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("n,G,tg,best,k", [(128, 1, 1, 1, 8), (128, 8, 4, 2, 8), (256, 8, 3, 1, 6), (60, 6, 2, 2, 5),
                                           (1, 1, 1, 1, 1), (33, 1, 1, 2, 33), (512, 32, 8, 2, 16), (1024, 16, 4, 2, 20),
                                           (1000, 1, 1, 1, 64), (7, 7, 3, 1, 3), (64, 32, 9, 2, 17), (513, 3, 2, 2, 4)])
def test_choice_weights_and_gradient(env, softmax, bias, n, G, tg, best, k):
    rng = np.random.default_rng([n, G, k, softmax, bias])
    for T, norm, scale, ld in ((1, True, 1.0, None), (37, False, 2.5, n + 3), (300, True, -0.5, None), (301, False, 1.0, n)):
        b = (rng.normal(size=n) * 0.05).astype(np.float32) if bias else None
        check(env, logits(rng, T, n), b, softmax, G, tg, best, k, norm, scale, ld, rng.normal(size=(T, k)))


@pytest.mark.parametrize("softmax", [True, False])
def test_choices_that_f32_cannot_tell_apart(env, softmax):
    """Scores a few units of 2^-26 from each other, in and across groups, and equal
    ones: the order is that of 64 bits."""
    rng = np.random.default_rng(11)
    T, n = 400, 128
    l = np.float32(1) + rng.integers(-3, 4, size=(T, n)).astype(np.float32) * np.float32(2.0 ** -23)
    b = (rng.integers(-2, 3, size=n) * 2.0 ** -26).astype(np.float32)
    for G, tg, best in ((1, 1, 1), (8, 4, 2), (8, 2, 1), (4, 3, 2)):
        check(env, l, b, softmax, G, tg, best, 8, True)
        check(env, l, b, softmax, G, tg, best, 20, False)
    few = np.full((T, n), -np.inf, np.float32)
    few[:, ::11] = l[:, ::11]  # fewer than a warp's candidates
    check(env, few, b, softmax, 1, 1, 1, 8, True)
    check(env, few, b, softmax, 8, 4, 2, 8, True)


@pytest.mark.parametrize("softmax", [True, False])
@pytest.mark.parametrize("n,G,tg,k", [(128, 8, 4, 8), (128, 8, 4, 16), (128, 32, 9, 8), (96, 8, 3, 5), (120, 5, 2, 8), (256, 16, 5, 8),
                                      (512, 8, 3, 7), (512, 8, 2, 16), (1024, 4, 2, 8), (1024, 32, 7, 20)])
def test_borders_between_groups_that_f32_cannot_tell(env, softmax, n, G, tg, k):
    """Groups that lead, groups that trail, and three at the border whose sums of two
    are some 2^-24 apart; and every group of a row at the border."""
    rng = np.random.default_rng([n, G, k])
    T, size = 200, n // G
    lead = np.argsort(rng.random((T, G)), axis=1)
    level = np.where(lead < tg - 2, 2.0, np.where(lead < tg + 1, 1.0, -1.0))  # three for two places
    l = np.repeat(level, size, axis=1) - 3 * rng.random((T, n))
    border = np.repeat((lead >= tg - 2) & (lead < tg + 1), size, axis=1)
    best = rng.random((T, G, size)).argsort(2).argsort(2).reshape(T, n) < min(3, size)  # three of each group near its top
    l = np.where(best & border, 1 + rng.integers(-3, 4, size=(T, n)) * 2.0 ** -23, l).astype(np.float32)
    b = (rng.integers(-2, 3, size=n) * 2.0 ** -26).astype(np.float32)
    for ld in (None, n + 1):
        check(env, l, b, softmax, G, tg, 2, k, True, ld=ld)
        check(env, l, b, softmax, G, tg, 1, k, True, ld=ld)
    l[l < 0.9] = -np.inf  # a group of less than two, and of none
    check(env, l, b, softmax, G, tg, 2, k, True)
    l = (1 + rng.integers(-3, 4, size=(T, n)) * 2.0 ** -23).astype(np.float32)
    check(env, l, b, softmax, G, tg, 2, k, True)


@pytest.mark.parametrize("softmax", [True, False])
@pytest.mark.parametrize("G,tg,best", [(1, 1, 1), (8, 4, 2)])
def test_equal_scores_go_to_the_lowest_expert(env, softmax, G, tg, best):
    n = 96 if G == 1 else 128
    for l in (np.zeros((5, n), np.float32), np.full((5, n), -3.0, np.float32)):
        for b in (None, np.zeros(n, np.float32), np.full(n, 0.25, np.float32)):
            check(env, l, b, softmax, G, tg, best, 8, True)
            check(env, l, b, softmax, G, tg, best, 30, True)


@pytest.mark.parametrize("softmax", [True, False])
@pytest.mark.parametrize("bias", [True, False])
def test_far_logits(env, softmax, bias):
    """Scores that underflow, a bias that chooses them, weights renormalised all the
    same; the largest and smallest logits."""
    rng = np.random.default_rng(5)
    T, n = 64, 64
    b = (rng.normal(size=n)).astype(np.float32) if bias else None
    l = (rng.normal(size=(T, n)) * 30 - 60).astype(np.float32)
    check(env, l, b, softmax, 1, 1, 1, 4, False)
    torch, smoe, dev = env
    for norm in (True, False):
        _, idx, w = route(env, l, b, softmax, 1, 1, 1, 4, norm, 1.0)
        ref = u.choose(l, b, softmax, 1, 1, 1, 4)
        assert (idx.cpu().numpy() == ref).all()
        if norm:
            x = np.take_along_axis(l.astype(np.float64), ref, 1)
            s = x - x.max(1, keepdims=True) if softmax else np.minimum(x, 0) - np.log1p(np.exp(-np.abs(x)))
            s = np.exp(s - s.max(1, keepdims=True))
            rw = s / s.sum(1, keepdims=True)
            # arguments of up to 200 are rounded here, 2^-24 of them
            assert (np.abs(w.cpu().numpy() - rw) <= 200 * 2.0 ** -22 * rw + 1e-30).all()
    if not softmax:
        l[:, 3] = np.inf
        l[:, 5] = np.float32(3e38)
        l[:, 7] = -np.float32(3e38)
        check(env, l, b, softmax, 1, 1, 1, 4, True)


@pytest.mark.parametrize("softmax", [True, False])
def test_rows_without_order_and_experts_that_are_off(env, softmax):
    torch, smoe, dev = env
    rng = np.random.default_rng(9)
    n, k = 32, 4
    l = logits(rng, 6, n, False)
    l[1, 7] = np.nan
    l[2] = -np.inf
    l[3, 1:] = -np.inf
    if softmax:
        l[4, 2] = np.inf
    _, idx, w = route(env, l, None, softmax, 4, 2, 2, k, True, 1.0)
    gi, gw = idx.cpu().numpy(), w.cpu().numpy()
    bad = [1, 4] if softmax else [1]
    assert (gi[bad] == np.arange(k)).all() and np.isnan(gw[bad]).all()
    assert (gi[2] == -1).all() and (gw[2] == 0).all()
    assert gi[3].tolist() == [0, -1, -1, -1] and gw[3].tolist() == [1, 0, 0, 0]
    fine = [t for t in range(6) if t not in bad]
    assert (gi[fine] == u.choose(l, None, softmax, 4, 2, 2, k)[fine]).all()
    # a bias of -inf turns an expert off, one that is NaN where it is on has no order
    b = np.zeros(n, np.float32)
    b[5] = -np.inf
    clean = logits(rng, 20, n, False)
    clean[:, 5] = 9
    check(env, clean, b, softmax, 1, 1, 1, k, True)
    check(env, clean, b, softmax, 4, 2, 2, k, False)
    b[6] = np.nan
    clean[3, 6] = -np.inf
    _, idx, w = route(env, clean, b, softmax, 1, 1, 1, k, True, 1.0)
    nan = np.isnan(w.cpu().numpy()).all(1)
    assert nan.sum() == 19 and not nan[3]


def test_gradient_of_lists_that_no_selection_makes(env):
    """Indices outside the experts count for nothing, an expert twice adds up."""
    torch, smoe, dev = env
    rng = np.random.default_rng(2)
    T, n, k = 9, 40, 40
    l = logits(rng, T, n, False)
    idx = rng.integers(-3, n + 3, size=(T, k)).astype(np.int32)
    idx[0, :] = 5
    dw = rng.normal(size=(T, k)).astype(np.float32)
    for softmax in (True, False):
        for norm in (True, False):
            there = (idx >= 0) & (idx < n)
            w = np.where(there, u.weights(l, np.where(there, idx, -1), softmax, norm, 1.0), 3.0).astype(np.float32)
            dl = torch.full((T, n), float("nan"), device=dev)
            smoe.smoe_route_rows_backward(torch.from_numpy(l).to(dev), T, n, n, int(not softmax), k, int(norm), 1.0,
                                          torch.from_numpy(idx).to(dev), torch.from_numpy(w).to(dev),
                                          torch.from_numpy(dw).to(dev), dl)
            d, mag = u.weights_gradient(l, idx, softmax, norm, 1.0, dw.astype(np.float64))
            bound = 4 * (rtol(n) + k * 2.0 ** -23) * (mag + np.abs(dw).sum(1, keepdims=True) * 2.0 ** -10)
            assert (np.abs(dl.cpu().numpy() - d) <= bound).all()


def test_many_rows_on_another_stream_in_a_graph(env):
    torch, smoe, dev = env
    rng = np.random.default_rng(1)
    T, n, k = 4097, 128, 8
    b = (rng.normal(size=n) * 0.05).astype(np.float32)
    L, B = torch.empty(T, n, device=dev), torch.from_numpy(b).to(dev)
    idx, w = torch.empty(T, k, dtype=torch.int32, device=dev), torch.empty(T, k, device=dev)
    dw, dl = torch.ones(T, k, device=dev), torch.empty(T, n, device=dev)
    s = torch.cuda.Stream()

    def calls():
        smoe.smoe_route_rows(L, T, n, n, B, smoe.SMOE_SCORE_SIGMOID, 8, 4, 2, k, 1, 2.5, idx, w, s)
        smoe.smoe_route_rows_backward(L, T, n, n, smoe.SMOE_SCORE_SIGMOID, k, 1, 2.5, idx, w, dw, dl, s)

    L.zero_()
    torch.cuda.synchronize()
    calls()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        calls()
    for _ in range(3):
        l = logits(rng, T, n)
        L.copy_(torch.from_numpy(l))
        g.replay()
        torch.cuda.synchronize()
        ref = u.choose(l, b, False, 8, 4, 2, k)
        assert (idx.cpu().numpy() == ref).all()
        rw = u.weights(l, ref, False, True, 2.5)
        assert (np.abs(w.cpu().numpy() - rw) <= rtol(n) * rw).all()
        d, mag = u.weights_gradient(l, ref, False, True, 2.5, np.ones((T, k)))
        assert (np.abs(dl.cpu().numpy() - d) <= 4 * (rtol(n) + k * 2.0 ** -23) * mag + 1e-36).all()
