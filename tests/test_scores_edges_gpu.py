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
