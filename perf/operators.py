"""Cases of the many-token mixture-of-experts operators: selecting experts for a
batch of tokens, sorting the tokens by expert and back (with their gradients),
and the products of 8-bit weights and activations, over one matrix and over the
experts of a sorted batch.

`run` is one pass of one operator: where `own` is true through the package's
entry points, elsewhere in elementary torch operations in 32 bits.
"""
import torch

own = False

# Sizes of the layer that the repository measures: router 128 x 4096, top 8;
# experts d_model 4096, d_ff 1536; the dense projection 8192 x 4096.


def listed():
    return [
        # a handful of tokens decoded together: the router's selection alone
        {"name": "select_small", "kind": "select", "T": 7, "E": 128, "k": 8, "masked": True, "grad": False},
        # a training batch's selection and the gradient to the logits, some
        # experts masked out and some padding tokens with no expert at all
        {"name": "select_train", "kind": "select", "T": 32768, "E": 128, "k": 8, "masked": True, "grad": True},
        # a decode batch's tokens brought to their experts
        {"name": "dispatch_small", "kind": "dispatch", "T": 16, "d": 4096, "E": 128, "k": 8, "dtype": "f32", "dropped": False},
        # a prefill's tokens, with padding tokens that go to no expert
        {"name": "dispatch_large", "kind": "dispatch", "T": 8191, "d": 4096, "E": 128, "k": 8, "dtype": "bf16", "dropped": True},
        # a training batch's gradient back from the experts' inputs
        {"name": "dispatch_grad", "kind": "dispatch_grad", "T": 2047, "d": 4096, "E": 128, "k": 8, "dtype": "f32", "dropped": True},
        # a decode batch's outputs weighted and summed
        {"name": "combine_small", "kind": "combine", "T": 16, "d": 4096, "E": 128, "k": 8, "dtype": "f32", "dropped": False},
        # a prefill's outputs
        {"name": "combine_large", "kind": "combine", "T": 4099, "d": 4096, "E": 128, "k": 8, "dtype": "f32", "dropped": True},
        # a training batch's gradient to the experts' outputs and the weights
        {"name": "combine_grad", "kind": "combine_grad", "T": 8191, "d": 4096, "E": 128, "k": 8, "dtype": "bf16", "dropped": True},
        # one decoded token through a dense projection
        {"name": "linear_one", "kind": "linear", "R": 1, "K": 4096, "N": 8192, "dtype": "f32"},
        # a prefill through the same projection, a ragged number of tokens
        {"name": "linear_batch", "kind": "linear", "R": 1999, "K": 4096, "N": 8192, "dtype": "bf16"},
        # a decode batch through one projection of the experts: most experts
        # get a row or two, some none
        {"name": "experts_small", "kind": "experts", "T": 16, "K": 4096, "N": 1536, "E": 128, "k": 8, "dtype": "bf16"},
        # a prefill through the same projection
        {"name": "experts_large", "kind": "experts", "T": 4096, "K": 4096, "N": 1536, "E": 128, "k": 8, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]."""
    import math
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _odd(rng, lo, hi):
    """An odd number so spread: sizes that no tile divides."""
    return min(_log(rng, lo, hi) | 1, (hi - 1) | 1)


def draw(rng):
    kind = rng.choice(["select", "dispatch", "dispatch_grad", "combine", "combine_grad", "linear", "experts"])
    if kind == "select":
        E = _log(rng, 8, 512)
        return {"kind": kind, "T": _odd(rng, 1, 32768), "E": E, "k": rng.randint(1, min(E, 16)),
                "masked": rng.random() < 0.5, "grad": rng.random() < 0.5}
    dtype = rng.choice(["f32", "bf16"])
    # rows of 16 bytes times an odd number (the 8-bit rows' alignment), outputs in any number
    if kind == "linear":
        return {"kind": kind, "R": _odd(rng, 1, 2048), "K": 16 * _odd(rng, 8, 512),
                "N": rng.choice([1, 4]) * _odd(rng, 100, 2048), "dtype": dtype}
    E = _log(rng, 4, 256)
    k = rng.randint(1, min(E, 8))
    if kind == "experts":
        return {"kind": kind, "T": _odd(rng, 1, 4096), "K": 16 * _odd(rng, 8, 256), "N": rng.choice([1, 4]) * _odd(rng, 50, 384),
                "E": min(E, 128), "k": min(k, 8), "dtype": dtype}
    d = rng.choice([1, 8]) * _odd(rng, 64, 512)
    return {"kind": kind, "T": _odd(rng, 1, 4096), "d": d, "E": E, "k": k, "dtype": dtype, "dropped": rng.random() < 0.5}


def _bytes(case):
    return 2 if case.get("dtype") == "bf16" else 4


def work(case):
    kind = case["kind"]
    e = _bytes(case)
    if kind == "select":
        T, E, k = case["T"], case["E"], case["k"]
        b = 4 * T * E + 8 * T * k
        f = 2 * T * E + 4 * T * k
        if case["grad"]:
            b += 4 * T * k + 4 * T * E
            f += 4 * T * k
        return {"bytes": b, "flops": f}
    if kind == "linear":
        R, K, N = case["R"], case["K"], case["N"]
        return {"bytes": e * R * K + N * K + 4 * N + e * R * N, "flops": 2 * R * N * K}
    T, k, E = case["T"], case["k"], case["E"]
    R = T * k
    if kind == "experts":
        K, N = case["K"], case["N"]
        used = E * (1 - (1 - 1 / E) ** R)  # experts with a row, were all equally likely
        return {"bytes": int(e * T * K + used * N * (K + 4) + 4 * R + e * R * N), "flops": 2 * R * N * K}
    d = case["d"]
    if kind == "dispatch":
        return {"bytes": 4 * R + e * T * d + 4 * (E + 1) + 8 * R + e * R * d, "flops": R}
    if kind == "dispatch_grad":
        return {"bytes": e * R * d + 4 * R + e * T * d, "flops": R * d}
    if kind == "combine":
        return {"bytes": e * R * d + 8 * R + e * T * d, "flops": 2 * R * d}
    return {"bytes": 2 * e * R * d + 12 * R + e * T * d, "flops": 3 * R * d}


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


def _select_plain(l, k):
    """Indices (-1: none left) and weights of each row's k largest."""
    v, i = torch.sort(l, dim=1, descending=True, stable=True)
    v, i = v[:, :k], i[:, :k]
    there = v > float("-inf")
    e = torch.where(there, torch.exp(v - torch.where(there[:, :1], v[:, :1], 0.0)), 0.0)
    s = e.sum(1, keepdim=True)
    return torch.where(there, i, -1).to(torch.int32), e / torch.where(s > 0, s, 1.0)


def _sort_plain(idx, E):
    """offsets, order, place of the slots of idx [T, k], sorted by expert."""
    a = idx.reshape(-1).long()
    key = torch.where((a >= 0) & (a < E), a, E)
    order = torch.argsort(key, stable=True)
    at = torch.empty_like(order)
    at[order] = torch.arange(a.numel(), device=a.device)
    offsets = torch.zeros(E + 1, dtype=torch.long, device=a.device)
    offsets[1:] = torch.cumsum((key[:, None] == torch.arange(E, device=a.device)).sum(0), 0)
    place = torch.where(key < E, at, -1 - at)
    return offsets.to(torch.int32), order.to(torch.int32), place.to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    kind = case["kind"]
    s = dict(case)
    if kind == "select":
        T, E, k = case["T"], case["E"], case["k"]
        s["logits"] = _logits(g, T, E, case["masked"])
        s["idx"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
        s["w"] = torch.empty(T, k, device="cuda")
        if case["grad"]:
            s["d_w"] = _randn(g, T, k)
            s["d_logits"] = torch.empty(T, E, device="cuda")
        return s
    dt = _dtype(case)
    if kind == "linear":
        R, K, N = case["R"], case["K"], case["N"]
        s["x"] = _randn(g, R, K, dtype=dt)
        s["x_src"] = R
    else:
        T, E, k = case["T"], case["E"], case["k"]
        idx, w = _select_plain(_logits(g, T, E, False), k)
        if case.get("dropped"):  # padding tokens: no expert at all; some single slots dropped
            off = torch.rand(T, 1, generator=g, device="cuda") < 1 / 32
            off = off | (torch.rand(T, k, generator=g, device="cuda") < 1 / 64)
            idx = torch.where(off, -1, idx)
        R = T * k
        s["idx"], s["top_w"] = idx, w
        offsets, order, place = _sort_plain(idx, E)
        if kind == "dispatch":
            s["x"] = _randn(g, T, case["d"], dtype=dt)
            s["offsets"], s["order"], s["place"] = torch.empty_like(offsets), torch.empty_like(order), torch.empty_like(place)
            s["xs"] = torch.empty(R, case["d"], dtype=dt, device="cuda")
            return s
        s["offsets"], s["order"], s["place"] = offsets, order, place
        if kind == "dispatch_grad":
            s["d_xs"] = _randn(g, R, case["d"], dtype=dt)
            s["d_x"] = torch.empty(T, case["d"], dtype=dt, device="cuda")
            return s
        if kind in ("combine", "combine_grad"):
            s["ys"] = _randn(g, R, case["d"], dtype=dt)
            if kind == "combine":
                s["out"] = torch.empty(T, case["d"], dtype=dt, device="cuda")
            else:
                s["d_out"] = _randn(g, T, case["d"], dtype=dt)
                s["d_ys"] = torch.empty(R, case["d"], dtype=dt, device="cuda")
                s["d_top_w"] = torch.empty(T, k, device="cuda")
            return s
        K, N = case["K"], case["N"]
        s["x"] = _randn(g, T, K, dtype=dt)
        s["x_src"] = T
        # the most rows of one expert, for the plain form's padded layout
        s["most"] = int((offsets[1:] - offsets[:-1]).max())
    n = case.get("E", 1) if kind == "experts" else 1
    s["wq"] = torch.randn(n * N, K, generator=g, device="cuda").mul_(32).round_().clamp_(-127, 127).to(torch.int8)
    s["w_scales"] = (0.5 + torch.rand(n * N, generator=g, device="cuda")) / (32 * K ** 0.5)
    s["xq"] = torch.empty(s["x_src"], K, dtype=torch.int8, device="cuda")
    s["x_scales"] = torch.empty(s["x_src"], device="cuda")
    s["y"] = torch.empty(R, N, dtype=dt, device="cuda")
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
    if kind == "select":
        smoe.smoe_topk_rows(s["logits"], s["T"], s["E"], s["E"], s["k"], s["idx"], s["w"])
        if not s["grad"]:
            return {"idx": s["idx"], "w": s["w"]}
        smoe.smoe_topk_rows_backward(s["idx"], s["w"], s["d_w"], s["T"], s["E"], s["k"], s["d_logits"])
        return {"idx": s["idx"], "w": s["w"], "d_logits": s["d_logits"]}
    code = _CODE[s["dtype"]]
    if kind == "dispatch":
        ws, need = s.get("ws"), s.get("need")
        if ws is None:
            ws, need = _workspace(s, smoe.smoe_dispatch_workspace_bytes(s["T"], s["k"], s["E"]))
        smoe.smoe_dispatch_tokens(s["idx"], s["T"], s["k"], s["E"], s["x"], code, s["d"], s["offsets"], s["order"],
                                  s["place"], s["xs"], ws, need)
        return {"offsets": s["offsets"], "order": s["order"], "place": s["place"], "xs": s["xs"]}
    if kind == "dispatch_grad":
        smoe.smoe_dispatch_tokens_backward(s["d_xs"], code, s["place"], s["T"], s["k"], s["d"], s["d_x"])
        return {"d_x": s["d_x"]}
    if kind == "combine":
        smoe.smoe_combine_tokens(s["ys"], code, s["place"], s["top_w"], s["T"], s["k"], s["d"], s["out"])
        return {"out": s["out"]}
    if kind == "combine_grad":
        smoe.smoe_combine_tokens_backward(s["d_out"], s["ys"], code, s["place"], s["top_w"], s["T"], s["k"], s["d"],
                                          s["d_ys"], s["d_top_w"])
        return {"d_ys": s["d_ys"], "d_top_w": s["d_top_w"]}
    smoe.smoe_quantize_rows_q8(s["x"], code, smoe.SMOE_Q8_PLAIN, s["x_src"], s["K"], s["xq"], s["x_scales"])
    ws, need = s.get("ws"), s.get("need")
    if kind == "linear":
        if ws is None:
            ws, need = _workspace(s, smoe.smoe_matmul_q8_workspace_bytes(s["R"], s["N"], s["K"]))
        smoe.smoe_matmul_q8(s["xq"], s["x_scales"], s["R"], s["wq"], s["w_scales"], s["N"], s["K"], s["y"], code, ws, need)
    else:
        if ws is None:
            ws, need = _workspace(s, smoe.smoe_experts_matmul_q8_workspace_bytes(
                s["T"], s["T"] * s["k"], s["E"], s["N"], s["K"]))
        smoe.smoe_experts_matmul_q8(s["xq"], s["x_scales"], s["T"], s["order"], s["k"], s["offsets"], s["T"] * s["k"],
                                    s["E"], s["wq"], s["w_scales"], s["N"], s["K"], s["y"], code, ws, need)
    return {"y": s["y"]}


# ---------------------------------------------------------------- the plain forms

def _quantize_plain(x):
    x = x.float()
    top = x.abs().amax(1, keepdim=True)
    up = torch.where(top > 0, torch.full_like(top, 127.0) / top, 0.0)
    return torch.round(x * up), top / torch.full_like(top, 127.0)


def run(state):
    if own:
        return _run_own(state)
    s = state
    kind = s["kind"]
    if kind == "select":
        idx, w = _select_plain(s["logits"], s["k"])
        if not s["grad"]:
            return {"idx": idx, "w": w}
        d = w * (s["d_w"] - (w * s["d_w"]).sum(1, keepdim=True))
        # slots without an expert have weight 0, hence gradient 0: adding them anywhere changes nothing
        d_logits = torch.zeros_like(s["logits"]).scatter_add_(1, idx.clamp(min=0).long(), d)
        return {"idx": idx, "w": w, "d_logits": d_logits}
    if kind == "linear":
        q, sx = _quantize_plain(s["x"])
        y = (q @ s["wq"].float().t()) * sx * s["w_scales"]
        return {"y": y.to(s["y"].dtype)}
    T, k = s["T"], s["k"]
    if kind == "dispatch":
        offsets, order, place = _sort_plain(s["idx"], s["E"])
        o = order.long()
        there = place[o] >= 0
        xs = torch.where(there[:, None], s["x"][o // k], 0)
        return {"offsets": offsets, "order": order, "place": place, "xs": xs}
    if kind == "experts":
        E, N, K, most = s["E"], s["N"], s["K"], s["most"]
        q, sx = _quantize_plain(s["x"])
        order, offsets = s["order"].long(), s["offsets"].long()
        row = torch.arange(T * k, device=order.device)
        e = torch.searchsorted(offsets[1:], row, right=True)
        at = e * most + row - offsets[e]  # the row's place in [E, most]
        padded = torch.zeros(E * most, K, device=order.device)
        padded[at] = q[order // k]
        y = torch.bmm(padded.view(E, most, K), s["wq"].view(E, N, K).float().transpose(1, 2)).view(E * most, N)[at]
        y = y * sx[order // k] * s["w_scales"].view(E, N)[e]
        return {"y": y.to(s["y"].dtype)}
    place = s["place"].long()
    there = place >= 0
    row = torch.where(there, place, -1 - place)  # a permutation of the rows
    if kind == "dispatch_grad":
        g = torch.where(there[:, None], s["d_xs"][row].float(), 0.0).view(T, k, -1).sum(1)
        return {"d_x": g.to(s["d_x"].dtype)}
    w = torch.where(there, s["top_w"].reshape(-1), 0.0)
    if kind == "combine":
        y = (s["ys"][row].float() * w[:, None]).view(T, k, -1).sum(1)
        return {"out": y.to(s["out"].dtype)}
    d_out = s["d_out"].float().repeat_interleave(k, 0)
    d_ys = torch.empty_like(s["ys"])
    d_ys[row] = (d_out * w[:, None]).to(d_ys.dtype)
    d_w = torch.where(there, (d_out * s["ys"][row].float()).sum(1), 0.0).view(T, k)
    return {"d_ys": d_ys, "d_top_w": d_w}


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """Token by token or expert by expert from the definitions, in float64.
    The quantised activations are defined by their float32 rounding (the scale
    and the reciprocal are float32 numbers), so that step is done in float32."""
    import numpy as np
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "select":
        l = s["logits"].double().cpu().numpy()
        T, E, k = case["T"], case["E"], case["k"]
        take = np.lexsort((np.broadcast_to(np.arange(E), (T, E)), -l), axis=1)[:, :k]
        v = np.take_along_axis(l, take, 1)
        w = np.exp(v - np.maximum(v[:, :1], -1e300))
        total = w.sum(1, keepdims=True)
        w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
        r = {"idx": None, "w": w}
        if case["grad"]:
            dw = s["d_w"].double().cpu().numpy()
            d = np.zeros((T, E))
            np.put_along_axis(d, take, w * (dw - np.einsum("tk,tk->t", w, dw)[:, None]), 1)
            r["d_logits"] = d
        return r
    if kind in ("linear", "experts"):
        x = s["x"].float().cpu().numpy()
        top = np.abs(x).max(1, keepdims=True)
        with np.errstate(divide="ignore", invalid="ignore"):
            inv = np.where(top > 0, np.float32(127) / top, np.float32(0))
        q = torch.from_numpy(np.rint(x * inv).astype(np.float64)).cuda()
        sx = torch.from_numpy((top / np.float32(127)).astype(np.float64)).cuda()
        sw = s["w_scales"].double()
        if kind == "linear":
            return {"y": torch.einsum("rk,nk->rn", q, s["wq"].double()) * sx * sw}
        E, N, k = case["E"], case["N"], case["k"]
        off = s["offsets"].tolist()
        y = torch.zeros(case["T"] * k, N, dtype=torch.float64, device="cuda")
        for e in range(E):
            a, b = off[e], off[e + 1]
            if b > a:
                t = torch.div(s["order"][a:b].long(), k, rounding_mode="floor")
                y[a:b] = torch.einsum("rk,nk->rn", q[t], s["wq"][e * N:(e + 1) * N].double()) * sx[t] * sw[e * N:(e + 1) * N]
        return {"y": y}
    T, k = case["T"], case["k"]
    if kind == "dispatch":
        o = s["idx"].reshape(-1).long().cpu().numpy()
        o = np.argsort(np.where(o < 0, case["E"], o), kind="stable")
        there = (s["idx"].reshape(-1).cpu().numpy()[o] >= 0).astype(np.float64)
        xs = s["x"][torch.from_numpy(o // k).cuda()].double() * torch.from_numpy(there).cuda()[:, None]
        return {"offsets": None, "order": None, "place": None, "xs": xs}
    place = s["place"].view(T, k).long()
    if kind == "dispatch_grad":
        d_x = torch.zeros(T, case["d"], dtype=torch.float64, device="cuda")
        for j in range(k):
            p = place[:, j]
            d_x += s["d_xs"][p.clamp(min=0)].double() * (p >= 0).double()[:, None]
        return {"d_x": d_x}
    w = s["top_w"].double()
    if kind == "combine":
        out = torch.zeros(T, case["d"], dtype=torch.float64, device="cuda")
        for j in range(k):
            p = place[:, j]
            out += s["ys"][p.clamp(min=0)].double() * ((p >= 0).double() * w[:, j])[:, None]
        return {"out": out}
    d_out = s["d_out"].double()
    d_ys = torch.zeros(T * k, case["d"], dtype=torch.float64, device="cuda")
    d_w = torch.zeros(T, k, dtype=torch.float64, device="cuda")
    for j in range(k):
        p = place[:, j]
        t = torch.nonzero(p >= 0).squeeze(1)
        d_ys[p[t]] = d_out[t] * w[t, j][:, None]
        d_w[t, j] = torch.einsum("td,td->t", d_out[t], s["ys"][p[t]].double())
    return {"d_ys": d_ys, "d_top_w": d_w}
