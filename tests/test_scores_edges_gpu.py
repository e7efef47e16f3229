"""Corners of the routing by scores against float64."""
import numpy as np
import pytest

import f8_util as u
import test_scores_gpu as t
from test_scores_gpu import env  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("softmax", [True, False])
@pytest.mark.parametrize("n,G,tg,k", [(8, 4, 1, 1), (128, 8, 4, 8), (128, 8, 4, 20), (96, 8, 3, 5), (512, 16, 5, 8), (1024, 4, 2, 20)])
def test_alike_experts_in_groups_of_different_numbers(env, softmax, n, G, tg, k):
    """Every expert that is on has one logit and one bias, and c is 0 in f32, or of the
    wrong sign: a group of one counts c, a group of two or more 2 c."""
    rng = np.random.default_rng([n, G, k])
    T, size = 60, n // G
    on = rng.integers(0, 4, size=(T, G))  # none, one, two, all
    on[0] = np.where(np.arange(G) < G // 2, 1, 3)
    on[1] = np.where(np.arange(G) < G // 2, 3, 1)
    place = rng.random((T, G, size)).argsort(2)
    there = (place < np.where(on == 3, size, np.minimum(on, size))[:, :, None]).reshape(T, n)
    for level in (-3.0, -88.0, -100.0, -120.0):
        l = np.where(there, np.float32(level), -np.inf).astype(np.float32)
        t.check(env, l, None, softmax, G, tg, 2, k, True)
        s = u.scores(np.full((1, n), level, np.float32), softmax)[0, 0]
        for b in (0.0, -np.float32(s), np.nextafter(-np.float32(s), np.float32(1))):
            t.check(env, l, np.full(n, b, np.float32), softmax, G, tg, 2, k, False)
            t.check(env, l, np.full(n, b, np.float32), softmax, G, tg, 1, k, False)


@pytest.mark.parametrize("softmax", [True, False])
@pytest.mark.parametrize("n,G,tg,k", [(128, 8, 4, 8), (128, 8, 4, 20), (60, 6, 2, 5), (256, 4, 2, 16), (1024, 32, 7, 20)])
def test_scores_that_64_bits_cannot_tell_apart(env, softmax, n, G, tg, k):
    """Without a bias the experts of the groups that stay are ordered by their logits:
    sigmoids of 40 and 41 are 1 in 64 bits, softmax terms far below the largest 0."""
    rng = np.random.default_rng([n, G, k, 1])
    T, size = 80, n // G
    # (the groups themselves are told apart by their two best)
    l = 40 + rng.integers(0, 64, size=(T, n)) * 0.125 if not softmax else -800 - rng.integers(0, 64, size=(T, n)) * 16.0
    level = rng.random((T, G)).argsort(1)
    head = np.repeat(level, size, axis=1) * 0.25 - (0 if softmax else 20)
    first = np.tile(np.arange(n) % size, (T, 1)) < 1  # one of each group far from the rest
    if softmax:
        l = np.where(first, head, l)
    else:
        l = np.where(np.repeat(level, size, axis=1) >= G - tg, l, head)
    l = l.astype(np.float32)
    l[rng.random((T, n)) < 0.02] = -np.inf
    p = u.scores(l, softmax)
    c = np.where(l == -np.inf, -np.inf, p)
    v = -np.sort(-c.reshape(T, G, size), axis=2)[:, :, :2]
    of = np.where(v[:, :, 0] > -np.inf, np.where(v > -np.inf, v, 0).sum(2), -np.inf)
    rank = np.argsort(np.argsort(-of, axis=1, kind="stable"), axis=1, kind="stable")
    left = np.where(np.repeat(rank < tg, size, axis=1), l, -np.inf)
    take = np.argsort(-left, axis=1, kind="stable")[:, :k]
    ref = np.where(np.take_along_axis(left, take, 1) > -np.inf, take, -1)
    _, idx, w = t.route(env, l, None, softmax, G, tg, 2, k, False, 1.0)
    gi = idx.cpu().numpy()
    assert (gi == ref).all(), np.argwhere(gi != ref)[:5]
    rw = u.weights(l, ref, softmax, False, 1.0)
    assert (np.abs(w.cpu().numpy() - rw) <= t.rtol(n) * rw + 1e-37).all()


@pytest.mark.parametrize("softmax", [True, False])
@pytest.mark.parametrize("low", [-np.finfo(np.float32).max, -3e38, 3e38, np.finfo(np.float32).max])
@pytest.mark.parametrize("n,G,tg,k", [(128, 8, 4, 8), (128, 8, 4, 20), (60, 6, 3, 7), (256, 4, 2, 16)])
def test_biases_whose_sum_of_two_leaves_f32(env, softmax, low, n, G, tg, k):
    """A mask of the type's lowest value is a bias like another: its experts come last,
    and a group of them counts less than any other that is on, but is not off."""
    rng = np.random.default_rng([n, G, k, 2])
    size = n // G
    l = t.logits(rng, 50, n, False)
    for some in (np.arange(n) // size >= 2, np.arange(n) % size > 1, rng.random(n) < 0.7, np.full(n, True)):
        b = np.where(some, np.float32(low), rng.normal(size=n) * 0.05).astype(np.float32)
        b[size] = -np.inf
        t.check(env, l, b, softmax, G, tg, 2, k, False)
        t.check(env, l, b, softmax, G, tg, 1, k, False)


@pytest.mark.parametrize("softmax", [True, False])
@pytest.mark.parametrize("scale", [3e38, -1e37, 2e-38])
@pytest.mark.parametrize("n,k", [(128, 8), (1000, 64), (7, 3)])
def test_scales_at_the_ends_of_f32(env, softmax, scale, n, k):
    """Renormalised weights are at most the scale, whatever the sum that they are over."""
    rng = np.random.default_rng([n, k])
    scale = float(np.float32(scale))
    l = np.concatenate([t.logits(rng, 20, n, False), t.logits(rng, 20, n, False) - 30]).astype(np.float32)
    L, idx, w = t.route(env, l, None, softmax, 1, 1, 1, k, True, scale)
    ref = u.choose(l, None, softmax, 1, 1, 1, k)
    assert (idx.cpu().numpy() == ref).all()
    rw = u.weights(l, ref, softmax, True, scale)
    gw = w.cpu().numpy().astype(np.float64)
    # below the normal numbers by a step of 2^-149
    assert (np.abs(gw - rw) <= t.rtol(n) * np.abs(rw) + 2.0 ** -148).all()
    torch, smoe, dev = env
    dw = (rng.random((40, k)) + 1).astype(np.float32)
    dl = torch.full((40, n), float("nan"), device=dev)
    smoe.smoe_route_rows_backward(L, 40, n, n, smoe.SMOE_SCORE_SOFTMAX if softmax else smoe.SMOE_SCORE_SIGMOID, k, 1, scale,
                                  idx, w, torch.from_numpy(dw).to(dev), dl)
    d, mag = u.weights_gradient(l, ref, softmax, True, scale, dw.astype(np.float64))
    got = dl.cpu().numpy().astype(np.float64)
    # a weight below the normal numbers is off by 2^-149, as a share by that over the scale
    share = (k + 2) * 2.0 ** -148 / abs(scale)
    assert (np.abs(got - d) <= 4 * (t.rtol(n) + k * 2.0 ** -23) * mag + 4 * share * mag.max() + 2.0 ** -147).all()
