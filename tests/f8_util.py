"""Plain float64 forms of the scored routing and of the 8-bit floating-point
operators, for the tests of both."""
import numpy as np


def scores(l, softmax):
    """[T, n] float64; 0 where the logit is -inf."""
    l = np.asarray(l, dtype=np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if not softmax:
            return 1 / (1 + np.exp(-l))
        top = l.max(1, keepdims=True)
        e = np.exp(l - np.where(top > -np.inf, top, 0))
        return e / np.maximum(e.sum(1, keepdims=True), 1e-320)


def choose(l, b, softmax, groups, top_groups, best, k):
    """Indices [T, k], -1 where no expert is left."""
    T, n = l.shape
    off = l == -np.inf
    c = scores(l, softmax)
    if b is not None:
        off = off | (b == -np.inf)
        c = c + np.where(b == -np.inf, 0, b).astype(np.float64)
    elif groups == 1 or best == 1:
        c = np.asarray(l, dtype=np.float64)  # the order of the scores, where those have run out of digits too
    c = np.where(off, -np.inf, c)
    if groups > 1:
        v = -np.sort(-c.reshape(T, groups, n // groups), axis=2)[:, :, :best]
        of = np.where(v[:, :, 0] > -np.inf, np.where(v > -np.inf, v, 0).sum(2), -np.inf)
        rank = np.argsort(np.argsort(-of, axis=1, kind="stable"), axis=1, kind="stable")
        c = np.where(np.repeat(rank < top_groups, n // groups, axis=1), c, -np.inf)
    take = np.argsort(-c, axis=1, kind="stable")[:, :k]
    return np.where(np.take_along_axis(c, take, 1) > -np.inf, take, -1)


def weights(l, idx, softmax, norm, scale):
    there = idx >= 0
    s = np.where(there, np.take_along_axis(scores(l, softmax), np.maximum(idx, 0), 1), 0)
    if norm:
        s = s / np.maximum(s.sum(1, keepdims=True), 1e-320)
    return s * scale


def weights_gradient(l, idx, softmax, norm, scale, dw):
    """(d_logits, a magnitude of its terms), [T, n] float64."""
    T, n = l.shape
    there = (idx >= 0) & (idx < n)
    at = np.where(there, idx, 0)
    w = np.where(there, weights(l, np.where(there, idx, -1), softmax, norm, scale), 0)
    dot, mag = (w * dw).sum(1, keepdims=True), np.abs(w * dw).sum(1, keepdims=True)
    g = w * dw - (w * dot / scale if norm else 0)
    m = np.abs(w * dw) + (np.abs(w) * mag / abs(scale) if norm else 0)  # magnitudes: w is negative where scale is
    p = scores(l, softmax)
    if not softmax:
        with np.errstate(over="ignore"):
            rest = 1 / (1 + np.exp(np.take_along_axis(np.asarray(l, np.float64), at, 1)))
        g, m = g * rest, m * rest
    d, dm = np.zeros((T, n)), np.zeros((T, n))
    for r in range(idx.shape[1]):
        t = np.nonzero(there[:, r])[0]
        np.add.at(d, (t, at[t, r]), g[t, r])
        np.add.at(dm, (t, at[t, r]), np.abs(m[t, r]))
    if softmax and not norm:
        d -= p * dot
        dm += p * mag
    return d, dm


def e4m3(codes):
    """float64 values of uint8 e4m3 codes (0x7f, 0xff: NaN)."""
    c = np.asarray(codes).astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((c & 0x7f) == 0x7f, np.nan, v)
    return np.where(c & 0x80, -v, v)


def to_e4m3(v):
    """Codes of float64 values of magnitude at most 448, nearest, ties to even."""
    table = e4m3(np.arange(0x7f))
    a = np.abs(np.asarray(v, dtype=np.float64))
    hi = np.clip(np.searchsorted(table, a), 1, 0x7e)
    lo = hi - 1
    up, down = table[hi] - a, a - table[lo]
    pick = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (pick | np.where(np.signbit(v), 0x80, 0)).astype(np.uint8)


def quantize(v):
    """(codes, scale) of a block of float32 values, by the float32 steps."""
    v = np.asarray(v, dtype=np.float32)
    top = np.abs(v).max() if v.size else np.float32(0)
    if not np.isfinite(top):
        return np.zeros(v.shape, np.uint8), np.float32(np.nan)
    if top == 0:
        return np.where(np.signbit(v), 0x80, 0).astype(np.uint8), np.float32(0)
    with np.errstate(over="ignore"):
        up = np.float32(448) / top
    if np.isinf(up):
        lift = np.float32(2.0 ** 64)
        return to_e4m3((v * lift) * (np.float32(448) / (top * lift))), top / np.float32(448)
    return to_e4m3((v * up).astype(np.float32)), top / np.float32(448)


def quantize_rows(v):
    """Blocks of 1 x 128 of [R, K] float32."""
    R, K = v.shape
    q, s = np.zeros((R, K), np.uint8), np.zeros((R, -(-K // 128)), np.float32)
    for r in range(R):
        for b in range(s.shape[1]):
            q[r, b * 128:b * 128 + 128], s[r, b] = quantize(v[r, b * 128:b * 128 + 128])
    return q, s


def spread(scales, axis, size):
    """A scale for each element along an axis, from one for each 128."""
    return np.take(np.repeat(scales, 128, axis), np.arange(size), axis)


def rows_of(q, s):
    return e4m3(q) * spread(s.astype(np.float64), 1, q.shape[1])


def weights_of(q, s):
    """[n, N, K] float64 of codes and scales [n, ceil(N / 128), ceil(K / 128)]."""
    return e4m3(q) * spread(spread(s.astype(np.float64), 1, q.shape[1]), 2, q.shape[2])
