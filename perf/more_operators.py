"""Cases of the operators of mixture-of-experts training and serving in 8-bit
floating point: routing by softmax or sigmoid scores with a bias and groups
(and its gradient), the quantisers to blocks of 128, the products of such rows
and weights over one matrix and over the experts of a sorted batch (their
gradient to the rows is the product with the transposed weights), and the
gradient of the experts' weights.

`run` is one pass of one operator: where `own` is true through the package's
entry points, elsewhere in elementary torch operations in 32 bits (the order of
the routing's scores in 64: scores next to each other decide which expert is
taken).
"""
import torch

own = False

# Sizes of the layer that the repository measures: router 128 x 4096, top 8;
# experts d_model 4096, d_ff 1536; the dense projection 8192 x 4096.


def listed():
    return [
        # a handful of tokens decoded together: the selection alone
        {"name": "route_small", "kind": "route", "T": 7, "E": 128, "score": "sigmoid", "bias": True, "groups": 8, "top_groups": 4,
         "best": 2, "k": 8, "norm": True, "masked": False, "grad": False},
        # a large prefill by groups of experts, with the bias that balances them
        {"name": "route_large", "kind": "route", "T": 32768, "E": 128, "score": "sigmoid", "bias": True, "groups": 8,
         "top_groups": 4, "best": 2, "k": 8, "norm": True, "masked": True, "grad": False},
        # a training batch: softmax over all experts, not renormalised, so that every expert's logit has a gradient
        {"name": "route_train", "kind": "route", "T": 16383, "E": 128, "score": "softmax", "bias": False, "groups": 1,
         "top_groups": 1, "best": 1, "k": 8, "norm": False, "masked": True, "grad": True},
        # the experts' hidden rows of a prefill, with their activation
        {"name": "quantize_act", "kind": "rows", "R": 32768, "K": 1536, "act": True, "dtype": "bf16"},
        # a layer's master weights after an update: codes for both directions
        {"name": "quantize_weights", "kind": "blocks", "n": 16, "N": 1536, "K": 4096, "dtype": "f32", "both": True},
        # one decoded token through a dense projection
        {"name": "linear_one", "kind": "linear", "R": 1, "K": 4096, "N": 8192, "dtype": "f32"},
        # a prefill through the same projection, a ragged number of tokens
        {"name": "linear_batch", "kind": "linear", "R": 1999, "K": 4096, "N": 8192, "dtype": "bf16"},
        # a decode batch through one projection of the experts: most experts
        # get a row or two, some none
        {"name": "experts_small", "kind": "experts", "T": 16, "K": 4096, "N": 1536, "E": 128, "k": 8, "dtype": "bf16", "sorted": False},
        # a prefill through the same projection
        {"name": "experts_large", "kind": "experts", "T": 4096, "K": 4096, "N": 1536, "E": 128, "k": 8, "dtype": "bf16", "sorted": False},
        # a training batch's gradient back through it: sorted rows, weights transposed
        {"name": "experts_back", "kind": "experts", "T": 2047, "K": 1536, "N": 4096, "E": 128, "k": 8, "dtype": "bf16", "sorted": True},
        # a small batch's gradient of a few experts' weights
        {"name": "weights_small", "kind": "weights", "T": 61, "K": 4096, "N": 1536, "E": 8, "k": 2, "dtype": "f32"},
        # a training batch's gradient of the projection's weights
        {"name": "weights_large", "kind": "weights", "T": 4096, "K": 4096, "N": 1536, "E": 128, "k": 8, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]."""
    import math
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _odd(rng, lo, hi):
    """An odd number so spread: sizes that no tile divides."""
    return min(_log(rng, lo, hi) | 1, (hi - 1) | 1)


def draw(rng):
    kind = rng.choice(["route", "route", "rows", "blocks", "linear", "linear", "experts", "experts", "weights"])
    if kind == "route":
        groups = rng.choice([1, 1, 2, 4, 6, 8])
        each = _log(rng, 4, 512 // groups)
        top = rng.randint(1, groups)
        return {"kind": kind, "T": _odd(rng, 1, 32768), "E": groups * each, "score": rng.choice(["softmax", "sigmoid"]),
                "bias": rng.random() < 0.5, "groups": groups, "top_groups": top, "best": rng.choice([1, 2]),
                "k": rng.randint(1, min(top * each, 16)), "norm": rng.random() < 0.5, "masked": rng.random() < 0.5,
                "grad": rng.random() < 0.5}
    dtype = rng.choice(["f32", "bf16"])
    if kind == "rows":
        return {"kind": kind, "R": _odd(rng, 1, 8192), "K": rng.choice([1, 8, 16]) * _odd(rng, 32, 512), "act": rng.random() < 0.5,
                "dtype": dtype}
    if kind == "blocks":
        return {"kind": kind, "n": _log(rng, 1, 8), "N": rng.choice([1, 16]) * _odd(rng, 32, 256),
                "K": rng.choice([1, 16]) * _odd(rng, 32, 256), "dtype": dtype, "both": rng.random() < 0.5}
    # rows of 16 bytes times an odd number (the 8-bit rows' alignment), outputs in any number
    if kind == "linear":
        return {"kind": kind, "R": _odd(rng, 1, 2048), "K": 16 * _odd(rng, 8, 512),
                "N": rng.choice([1, 4]) * _odd(rng, 100, 2048), "dtype": dtype}
    E = _log(rng, 4, 128)
    k = rng.randint(1, min(E, 8))
    if kind == "experts":
        return {"kind": kind, "T": _odd(rng, 1, 4096), "K": 16 * _odd(rng, 8, 256), "N": rng.choice([1, 4]) * _odd(rng, 50, 384),
                "E": E, "k": k, "dtype": dtype, "sorted": rng.random() < 0.5}
    # rows of 16 bytes in bf16
    return {"kind": kind, "T": _odd(rng, 1, 4096), "K": 8 * _odd(rng, 8, 256), "N": 8 * _odd(rng, 8, 128),
            "E": min(E, 64), "k": k, "dtype": dtype}


def _e(case):
    return 2 if case.get("dtype") == "bf16" else 4


def _up(a, b):
    return -(-a // b)


def work(case):
    kind = case["kind"]
    if kind == "route":
        T, E, k = case["T"], case["E"], case["k"]
        b = 4 * T * E + 8 * T * k + (4 * E if case["bias"] else 0)
        f = 4 * T * E + 4 * T * k
        if case["grad"]:
            b += 4 * T * k + 4 * T * E
            f += 2 * T * E
        return {"bytes": b, "flops": f}
    e = _e(case)
    if kind == "rows":
        R, K = case["R"], case["K"]
        return {"bytes": R * K * (e * (2 if case["act"] else 1) + 1) + 4 * R * _up(K, 128), "flops": R * K * (8 if case["act"] else 3)}
    if kind == "blocks":
        n, N, K = case["n"], case["N"], case["K"]
        two = 2 if case["both"] else 1
        return {"bytes": n * (N * K * (e + two) + 4 * two * _up(N, 128) * _up(K, 128)), "flops": 3 * n * N * K}
    K, N = case["K"], case["N"]
    if kind == "linear":
        R = case["R"]
        return {"bytes": R * K + 4 * R * _up(K, 128) + N * K + 4 * _up(N, 128) * _up(K, 128) + e * R * N, "flops": 2 * R * N * K}
    T, k, E = case["T"], case["k"], case["E"]
    R = T * k
    if kind == "experts":
        used = E * (1 - (1 - 1 / E) ** R)  # experts with a row, were all equally likely
        src = R if case["sorted"] else T
        return {"bytes": int(src * (K + 4 * _up(K, 128)) + used * (N * K + 4 * _up(N, 128) * _up(K, 128)) + 4 * R + e * R * N),
                "flops": 2 * R * N * K}
    return {"bytes": 2 * R * (N + K) + e * E * N * K, "flops": 2 * R * N * K}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _logits(g, T, E, masked):
    """Router logits: some experts are more popular than others (a
    standard deviation of 0.25 beside each token's own 1); masked: about
    one logit in ten is -inf (an expert that is off for the token) and one
    token in sixteen has none left (padding)."""
    l = _randn(g, T, E) + 0.25 * _randn(g, 1, E)
    if masked:
        off = torch.rand(T, E, generator=g, device="cuda") < 0.1
        off |= torch.rand(T, 1, generator=g, device="cuda") < 1 / 16
        l = torch.where(off, torch.full_like(l, float("-inf")), l)
    return l


def _codes(g, *shape):
    """e4m3 codes of normal values that use the type's whole range."""
    return torch.randn(*shape, generator=g, device="cuda").mul_(100).clamp_(-448, 448).to(torch.float8_e4m3fn)


def _sorted_batch(g, T, k, E):
    """offsets [E + 1] and order [T k] of a batch whose experts are not
    equally popular, its slots sorted by expert."""
    idx = torch.topk(_logits(g, T, E, False), k, dim=1).indices.reshape(-1)
    order = torch.argsort(idx, stable=True)
    count = torch.zeros(E, dtype=torch.long, device="cuda").index_add_(0, idx, torch.ones_like(idx))
    offsets = torch.zeros(E + 1, dtype=torch.long, device="cuda")
    offsets[1:] = torch.cumsum(count, 0)
    return offsets.to(torch.int32), order.to(torch.int32), int(count.max())


def prepare(case, seed):
    g = _gen(seed)
    kind = case["kind"]
    s = dict(case)
    empty = lambda *shape, dtype=torch.float32: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    f8 = torch.float8_e4m3fn
    if kind == "route":
        T, E, k = case["T"], case["E"], case["k"]
        s["logits"] = _logits(g, T, E, case["masked"])
        # as the balancing has moved it: a few hundredths of a sigmoid, a few thousandths of a softmax
        s["b"] = _randn(g, E) * (0.05 if case["score"] == "sigmoid" else 0.005) if case["bias"] else None
        s["idx"], s["w"] = empty(T, k, dtype=torch.int32), empty(T, k)
        if case["grad"]:
            s["d_w"], s["d_logits"] = _randn(g, T, k), empty(T, E)
        return s
    dt = _dtype(case)
    if kind == "rows":
        R, K = case["R"], case["K"]
        # rows and columns of different size, as activations have them
        s["x"] = (torch.randn(R, K * (2 if case["act"] else 1), generator=g, device="cuda")
                  * torch.exp(_randn(g, R, 1))).to(dt)
        s["q"], s["scales"] = empty(R, K, dtype=f8), empty(R, _up(K, 128))
        return s
    if kind == "blocks":
        n, N, K = case["n"], case["N"], case["K"]
        s["x"] = (torch.randn(n, N, K, generator=g, device="cuda") / K ** 0.5).to(dt)
        s["q"], s["scales"] = empty(n, N, K, dtype=f8), empty(n, _up(N, 128), _up(K, 128))
        if case["both"]:
            s["qt"], s["scales_t"] = empty(n, K, N, dtype=f8), empty(n, _up(K, 128), _up(N, 128))
        return s
    K, N = case["K"], case["N"]
    if kind == "weights":
        T, k, E = case["T"], case["k"], case["E"]
        s["offsets"], _, s["most"] = _sorted_batch(g, T, k, E)
        s["xs"], s["d_ys"] = _randn(g, T * k, K, dtype=torch.bfloat16), _randn(g, T * k, N, dtype=torch.bfloat16)
        s["d_w"] = empty(E, N, K, dtype=dt)
        return s
    if kind == "linear":
        n, R, src = 1, case["R"], case["R"]
    else:
        T, k, n = case["T"], case["k"], case["E"]
        R = T * k
        s["offsets"], s["order"], s["most"] = _sorted_batch(g, T, k, n)
        src = R if case["sorted"] else T
    s["src"] = src
    s["xq"], s["x_scales"] = _codes(g, src, K), (0.5 + torch.rand(src, _up(K, 128), generator=g, device="cuda")) / 100
    s["wq"] = _codes(g, n * N, K).view(n, N, K)
    s["w_scales"] = (0.5 + torch.rand(n, _up(N, 128), _up(K, 128), generator=g, device="cuda")) / (100 * K ** 0.5)
    s["y"] = empty(R, N, dtype=dt)
    return s


# ---------------------------------------------------------------- the framework's operators

_CODE = {"f32": 0, "bf16": 1}


def _workspace(s, need):
    """The state's workspace, made by its first pass and kept, as a program keeps it."""
    if "ws" not in s:
        s["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
        s["need"] = need
    return s["ws"], s["need"]


def _run_own(s):
    import moe_expert_ffn_smoe_gb300 as smoe
    kind = s["kind"]
    if kind == "route":
        score = smoe.SMOE_SCORE_SIGMOID if s["score"] == "sigmoid" else smoe.SMOE_SCORE_SOFTMAX
        smoe.smoe_route_rows(s["logits"], s["T"], s["E"], s["E"], s["b"], score, s["groups"], s["top_groups"], s["best"], s["k"],
                             int(s["norm"]), 1.0, s["idx"], s["w"])
        if not s["grad"]:
            return {"idx": s["idx"], "w": s["w"]}
        smoe.smoe_route_rows_backward(s["logits"], s["T"], s["E"], s["E"], score, s["k"], int(s["norm"]), 1.0, s["idx"], s["w"],
                                      s["d_w"], s["d_logits"])
        return {"idx": s["idx"], "w": s["w"], "d_logits": s["d_logits"]}
    code = _CODE[s["dtype"]]
    if kind == "rows":
        smoe.smoe_quantize_rows_f8(s["x"], code, smoe.SMOE_Q8_SILU_MUL if s["act"] else smoe.SMOE_Q8_PLAIN, s["R"], s["K"], s["q"],
                                   s["scales"])
        return {"q": s["q"], "scales": s["scales"]}
    if kind == "blocks":
        smoe.smoe_quantize_blocks_f8(s["x"], code, s["n"], s["N"], s["K"], s["q"], s["scales"], s.get("qt"), s.get("scales_t"))
        return {n: s[n] for n in ("q", "scales", "qt", "scales_t") if n in s}
    if kind == "weights":
        smoe.smoe_experts_weight_grad(s["d_ys"], s["xs"], s["offsets"], s["T"] * s["k"], s["E"], s["N"], s["K"], 0, s["d_w"], code)
        return {"d_w": s["d_w"]}
    ws, need = s.get("ws"), s.get("need")
    if kind == "linear":
        if ws is None:
            ws, need = _workspace(s, smoe.smoe_matmul_f8_workspace_bytes(s["R"], s["N"], s["K"]))
        smoe.smoe_matmul_f8(s["xq"], s["x_scales"], s["R"], s["wq"], s["w_scales"], s["N"], s["K"], s["y"], code, ws, need)
    else:
        if ws is None:
            ws, need = _workspace(s, smoe.smoe_experts_matmul_f8_workspace_bytes(s["src"], s["T"] * s["k"], s["E"], s["N"], s["K"]))
        smoe.smoe_experts_matmul_f8(s["xq"], s["x_scales"], s["src"], None if s["sorted"] else s["order"], s["k"], s["offsets"],
                                    s["T"] * s["k"], s["E"], s["wq"], s["w_scales"], s["N"], s["K"], s["y"], code, ws, need)
    return {"y": s["y"]}


# ---------------------------------------------------------------- the plain forms

def _scores(l, score):
    """Scores of logits, 0 where the logit is -inf (a row of nothing else too)."""
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    top = l.amax(1, keepdim=True)
    e = torch.exp(l - torch.where(top > float("-inf"), top, 0.0))
    total = e.sum(1, keepdim=True)
    return e / torch.where(total > 0, total, 1.0)


def _choose(l, s):
    """Indices [T, k] of the experts of each row (-1: none left), by the scores in 64 bits."""
    T, E, G = s["T"], s["E"], s["groups"]
    off = l == float("-inf")
    c = _scores(l.double(), s["score"])
    if s["b"] is not None:
        c = c + s["b"].double()
    c = torch.where(off, float("-inf"), c)
    if G > 1:
        best = torch.sort(c.view(T, G, E // G), dim=2, descending=True).values[:, :, :s["best"]]
        there = best > float("-inf")
        of = torch.where(there, best, 0.0).sum(2)
        of = torch.where(there[:, :, 0], of, float("-inf"))
        taken = torch.sort(of, dim=1, descending=True, stable=True).indices[:, :s["top_groups"]]
        inside = torch.zeros(T, G, dtype=torch.bool, device=l.device).scatter_(1, taken, True)
        c = torch.where(inside.repeat_interleave(E // G, 1), c, float("-inf"))
    v, i = torch.sort(c, dim=1, descending=True, stable=True)
    v, i = v[:, :s["k"]], i[:, :s["k"]]
    return torch.where(v > float("-inf"), i, -1)


def _blocks_up(scales, dim, times, size):
    return torch.repeat_interleave(scales, times, dim).narrow(dim, 0, size)


def _padded(x, cols, to):
    return torch.cat([x, x.new_zeros(*x.shape[:-1], to - cols)], -1) if to > cols else x


def _to_codes(v, top):
    """Codes of v (in 32 bits) where `top` is its block's largest magnitude, and the scale."""
    up = torch.where(top > 0, torch.full_like(top, 448.0) / top, 0.0)
    return (v * up).clamp(-448, 448).to(torch.float8_e4m3fn), top / torch.full_like(top, 448.0)


def _batch(s, a):
    """Rows of a sorted batch as [E, most, cols], zeros behind each expert's."""
    E, most, offsets = s["E"], s["most"], s["offsets"].long()
    row = torch.arange(a.shape[0], device=a.device)
    e = torch.searchsorted(offsets[1:], row, right=True)
    at = e * most + row - offsets[e]
    padded = torch.zeros(E * most, a.shape[1], device=a.device)
    padded[at] = a
    return padded.view(E, most, -1), at


def run(state):
    if own:
        return _run_own(state)
    s = state
    kind = s["kind"]
    if kind == "route":
        l = s["logits"]
        idx = _choose(l, s)
        there = idx >= 0
        at = idx.clamp(min=0)
        p = _scores(l, s["score"])
        v = torch.where(there, p.gather(1, at), 0.0)
        total = v.sum(1, keepdim=True)
        w = v / torch.where(total > 0, total, 1.0) if s["norm"] else v
        if not s["grad"]:
            return {"idx": idx.to(torch.int32), "w": w}
        d = w * s["d_w"]
        if s["norm"]:
            d = d - w * d.sum(1, keepdim=True)
        if s["score"] == "sigmoid":
            d = torch.where(there, d / (1 + torch.exp(l.gather(1, at))), 0.0)
        d_logits = torch.zeros_like(l).scatter_add_(1, at, d)
        if s["score"] == "softmax" and not s["norm"]:
            d_logits = d_logits - p * d.sum(1, keepdim=True)
        return {"idx": idx.to(torch.int32), "w": w, "d_logits": d_logits}
    if kind == "rows":
        K = s["K"]
        v = s["x"].float()
        if s["act"]:
            v = v[:, :K] / (1 + torch.exp(-v[:, :K])) * v[:, K:]
        v = _padded(v, K, _up(K, 128) * 128).view(s["R"], -1, 128)
        q, scales = _to_codes(v, v.abs().amax(2, keepdim=True))
        return {"q": q.view(s["R"], -1)[:, :K], "scales": scales.view(s["R"], -1)}
    if kind == "blocks":
        n, N, K = s["n"], s["N"], s["K"]
        nb, kb = _up(N, 128), _up(K, 128)
        v = _padded(s["x"].float(), K, kb * 128)
        v = _padded(v.transpose(1, 2), N, nb * 128).transpose(1, 2).reshape(n, nb, 128, kb, 128)
        q, scales = _to_codes(v, v.abs().amax((2, 4), keepdim=True))
        q, scales = q.view(n, nb * 128, kb * 128)[:, :N, :K], scales.view(n, nb, kb)
        r = {"q": q, "scales": scales}
        if s["both"]:
            r["qt"], r["scales_t"] = q.transpose(1, 2).contiguous(), scales.transpose(1, 2).contiguous()
        return r
    if kind == "weights":
        x, _ = _batch(s, s["xs"].float())
        d, _ = _batch(s, s["d_ys"].float())
        return {"d_w": torch.bmm(d.transpose(1, 2), x).to(s["d_w"].dtype)}
    K, N = s["K"], s["N"]
    x = s["xq"].float() * _blocks_up(s["x_scales"], 1, 128, K)
    w = s["wq"].float() * _blocks_up(_blocks_up(s["w_scales"], 1, 128, N), 2, 128, K)
    if kind == "linear":
        y = x @ w[0].t()
    else:
        x, at = _batch(s, x if s["sorted"] else x[s["order"].long() // s["k"]])
        y = torch.bmm(x, w.transpose(1, 2)).view(-1, N)[at]
    return {"y": y.to(s["y"].dtype)}


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """Row by row or expert by expert from the definitions, in float64.  Codes
    are defined by their float32 steps, so the quantisers' have no such value;
    their scales have."""
    import numpy as np
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "route":
        T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
        l = s["logits"].double().cpu().numpy()
        on = np.isfinite(l)
        with np.errstate(over="ignore"):
            if case["score"] == "sigmoid":
                p = 1 / (1 + np.exp(-l))
            else:
                p = np.exp(l - np.where(on.any(1), l.max(1), 0.0)[:, None])
                p /= np.maximum(p.sum(1), 1e-300)[:, None]
            c = np.where(on, p if s["b"] is None else p + s["b"].double().cpu().numpy(), -np.inf)
            if G > 1:
                b = -np.sort(-c.reshape(T, G, E // G), axis=2)[:, :, :case["best"]]
                of = np.where(np.isfinite(b[:, :, 0]), np.where(np.isfinite(b), b, 0).sum(2), -np.inf)
                rank = np.argsort(np.argsort(-of, axis=1, kind="stable"), axis=1, kind="stable")
                c = np.where(np.repeat(rank < case["top_groups"], E // G, axis=1), c, -np.inf)
            take = np.argsort(-c, axis=1, kind="stable")[:, :k]
            there = np.isfinite(np.take_along_axis(c, take, 1))
            w = np.where(there, np.take_along_axis(p, take, 1), 0)
            if case["norm"]:
                w = w / np.maximum(w.sum(1, keepdims=True), 1e-300)
            r = {"idx": None, "w": w}
            if case["grad"]:
                d = w * s["d_w"].double().cpu().numpy()
                if case["norm"]:
                    d = d - w * d.sum(1, keepdims=True)
                if case["score"] == "sigmoid":
                    d = np.where(there, d / (1 + np.exp(np.take_along_axis(l, take, 1))), 0)
                full = np.zeros((T, E))
                np.put_along_axis(full, take, d, 1)
                if case["score"] == "softmax" and not case["norm"]:
                    full -= p * d.sum(1, keepdims=True)
                r["d_logits"] = full
        return r
    K = case["K"]
    if kind == "rows":
        v = s["x"].double()
        if case["act"]:
            v = torch.sigmoid(v[:, :K]) * v[:, :K] * v[:, K:]
        tops = [v[:, c:c + 128].abs().amax(1) for c in range(0, K, 128)]
        return {"q": None, "scales": torch.stack(tops, 1) / 448}
    N = case["N"]
    if kind == "blocks":
        x = s["x"].abs()
        tops = torch.stack([torch.stack([x[:, r:r + 128, c:c + 128].amax((1, 2)).double() for c in range(0, K, 128)], 1)
                            for r in range(0, N, 128)], 1) / 448
        r = {"q": None, "scales": tops}
        if case["both"]:
            r["qt"], r["scales_t"] = None, tops.transpose(1, 2)
        return r
    if kind == "weights":
        at = s["offsets"].tolist()
        return {"d_w": torch.stack([torch.einsum("rn,rk->nk", s["d_ys"][a:b].double(), s["xs"][a:b].double())
                                    for a, b in zip(at[:-1], at[1:])])}
    nb, kb = torch.arange(N, device="cuda") // 128, torch.arange(K, device="cuda") // 128
    x = s["xq"].double() * s["x_scales"].double()[:, kb]
    if kind == "linear":
        return {"y": torch.einsum("rk,nk->rn", x, s["wq"][0].double() * s["w_scales"][0].double()[nb][:, kb])}
    at, k = s["offsets"].tolist(), case["k"]
    y = torch.zeros(case["T"] * k, N, dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        a, b = at[e], at[e + 1]
        if b > a:
            rows = x[a:b] if case["sorted"] else x[torch.div(s["order"][a:b].long(), k, rounding_mode="floor")]
            y[a:b] = torch.einsum("rk,nk->rn", rows, s["wq"][e].double() * s["w_scales"][e].double()[nb][:, kb])
    return {"y": y}
