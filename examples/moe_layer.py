"""A mixture-of-experts layer for a batch of tokens on the many-token calls.

* ``Q8Layer``: serving.  Router, the tokens sorted by expert, gate/up and down
  products with 8-bit weights and activations, the weighted sum back: eight
  calls, nothing read back to the host, so that the whole layer can be
  captured in one CUDA graph.
* ``top_k``, ``dispatch``, ``combine``: the same routing under torch's
  autograd (each backward is the library's own call, and has none of its own:
  a second gradient is refused), for training experts written in torch.

``python examples/moe_layer.py`` runs both on a GPU with seeded weights.
"""
import contextlib
import os
import sys

import torch
from torch.autograd.function import once_differentiable

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_expert_ffn_smoe_gb300 as smoe  # noqa: E402

_CODE = {torch.float32: smoe.SMOE_F32, torch.bfloat16: smoe.SMOE_BF16}


def _check(name, t, shape, dtypes):
    """t is a GPU tensor of `shape` (None: any length) and of one of `dtypes`:
    the library takes addresses, and what it is handed wrongly it reads wrongly."""
    if t.dtype not in dtypes:
        raise TypeError(f"{name} is {t.dtype}, not " + " or ".join(map(str, dtypes)))
    if not t.is_cuda:
        raise ValueError(f"{name} is on {t.device}, not on a GPU")
    if t.dim() != len(shape) or any(w is not None and w != n for n, w in zip(t.shape, shape)):
        raise ValueError(f"{name} has the shape {tuple(t.shape)}, not {shape}")


_FLOATS = (torch.float32, torch.bfloat16, torch.float16, torch.float64)
_INTS = (torch.int32, torch.int64, torch.int16, torch.int8, torch.uint8)


def _bytes(n, device):
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device)


def quantize_weights(w):
    """int8 codes and one scale per output row of w [..., n_out, n_in]."""
    _check("w", w, (None,) * w.dim(), tuple(_CODE))
    q = torch.empty(w.shape, dtype=torch.int8, device=w.device)
    scales = torch.empty(w.shape[:-1], device=w.device)
    rows = w.numel() // w.shape[-1]
    smoe.smoe_quantize_rows_q8(w.contiguous(), _CODE[w.dtype], smoe.SMOE_Q8_PLAIN, rows, w.shape[-1], q, scales)
    return q, scales


class Q8Layer:
    """n_experts experts of d_model -> d_ff -> d_model in 8 bits, top-k routed,
    for up to max_tokens tokens a call.

    gate: router weights bf16 [n_experts, d_model] (bit patterns, int16);
    gate_up: [n_experts, 2 d_ff, d_model], the gate rows first, and
    down: [n_experts, d_model, d_ff], f32 or bf16, quantised here."""

    def __init__(self, gate, gate_up, down, k, max_tokens):
        n, d, d_ff = *gate.shape, down.shape[-1]
        _check("gate", gate, (n, d), (torch.int16, torch.bfloat16))
        _check("gate_up", gate_up, (n, 2 * d_ff, d), tuple(_CODE))
        _check("down", down, (n, d, d_ff), tuple(_CODE))
        dev, gate, self.max_tokens = gate.device, gate.contiguous(), max_tokens
        self.gate, self.gate32, self.k = gate, gate.view(torch.bfloat16).float(), k
        self.n, self.d_ff, self.d = gate_up.shape[0], down.shape[2], down.shape[1]
        self.gu, self.gu_scales = quantize_weights(gate_up)
        self.dn, self.dn_scales = quantize_weights(down)
        rows = max_tokens * k
        f32 = lambda *s: torch.empty(*s, device=dev)  # noqa: E731
        i32 = lambda *s: torch.empty(*s, dtype=torch.int32, device=dev)  # noqa: E731
        i8 = lambda *s: torch.empty(*s, dtype=torch.int8, device=dev)  # noqa: E731
        bf = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device=dev)  # noqa: E731
        self.logits, self.idx, self.w = f32(max_tokens, self.n), i32(max_tokens, k), f32(max_tokens, k)
        self.offsets, self.order, self.place = i32(self.n + 1), i32(rows), i32(rows)
        self.xq, self.x_scales = i8(max_tokens, self.d), f32(max_tokens)
        self.h, self.hq, self.h_scales = bf(rows, 2 * self.d_ff), i8(rows, self.d_ff), f32(rows)
        self.ys = bf(rows, self.d)
        need = max(smoe.smoe_dispatch_workspace_bytes(max_tokens, k, self.n),
                   smoe.smoe_experts_matmul_q8_workspace_bytes(max_tokens, rows, self.n, 2 * self.d_ff, self.d),
                   smoe.smoe_experts_matmul_q8_workspace_bytes(rows, rows, self.n, self.d, self.d_ff))
        self.ws = _bytes(need, dev)
        self.need = need

    def __call__(self, x, out, stream=None):
        """out[t] (bf16) = the layer's output for x[t] (f32 [tokens, d_model]),
        both contiguous."""
        _check("x", x, (None, self.d), (torch.float32,))
        _check("out", out, (x.shape[0], self.d), (torch.bfloat16,))
        if x.shape[0] > self.max_tokens:
            raise ValueError(f"{x.shape[0]} tokens, where the layer was made for {self.max_tokens}")
        if not (x.is_contiguous() and out.is_contiguous()):
            raise ValueError("x and out are to be contiguous")
        T, k, n, d, ff = x.shape[0], self.k, self.n, self.d, self.d_ff
        R = T * k
        if T <= 64 and n % 4 == 0:  # a matvec writes to 16-byte boundaries
            smoe.matvec_bf16_batch([self.gate] * T, [x.data_ptr() + 4 * d * t for t in range(T)],
                                   [self.logits.data_ptr() + 4 * n * t for t in range(T)], [n] * T, [d] * T, stream)
        else:  # a matvec a token would read the router's weights T times
            with torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext():
                torch.mm(x, self.gate32.t(), out=self.logits[:T])
        smoe.smoe_topk_rows(self.logits, T, n, n, k, self.idx, self.w, stream)
        smoe.smoe_dispatch_tokens(self.idx, T, k, n, None, smoe.SMOE_F32, 0, self.offsets, self.order, self.place, None,
                                  self.ws, self.need, stream)
        smoe.smoe_quantize_rows_q8(x, smoe.SMOE_F32, smoe.SMOE_Q8_PLAIN, T, d, self.xq, self.x_scales, stream)
        smoe.smoe_experts_matmul_q8(self.xq, self.x_scales, T, self.order, k, self.offsets, R, n, self.gu, self.gu_scales,
                                    2 * ff, d, self.h, smoe.SMOE_BF16, self.ws, self.need, stream)
        smoe.smoe_quantize_rows_q8(self.h, smoe.SMOE_BF16, smoe.SMOE_Q8_SILU_MUL, R, ff, self.hq, self.h_scales, stream)
        smoe.smoe_experts_matmul_q8(self.hq, self.h_scales, R, None, 1, self.offsets, R, n, self.dn, self.dn_scales, d, ff,
                                    self.ys, smoe.SMOE_BF16, self.ws, self.need, stream)
        smoe.smoe_combine_tokens(self.ys, smoe.SMOE_BF16, self.place, self.w, T, k, d, out, stream)
        return out


class _TopK(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k):
        logits = logits.contiguous()
        T, n = logits.shape
        idx = torch.empty(T, k, dtype=torch.int32, device=logits.device)
        w = torch.empty(T, k, device=logits.device)
        smoe.smoe_topk_rows(logits, T, n, n, k, idx, w)
        ctx.save_for_backward(idx, w)
        ctx.n = n
        ctx.mark_non_differentiable(idx)
        return idx, w

    @staticmethod
    @once_differentiable
    def backward(ctx, _, d_w):
        idx, w = ctx.saved_tensors
        T, k = idx.shape
        d = torch.empty(T, ctx.n, device=w.device)
        smoe.smoe_topk_rows_backward(idx, w, d_w.contiguous(), T, ctx.n, k, d)
        return d, None


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, idx, n):
        x, idx = x.contiguous(), idx.contiguous()
        T, k = idx.shape
        i32 = lambda m: torch.empty(m, dtype=torch.int32, device=x.device)  # noqa: E731
        offsets, order, place = i32(n + 1), i32(T * k), i32(T * k)
        xs = torch.empty(T * k, x.shape[1], dtype=x.dtype, device=x.device)
        need = smoe.smoe_dispatch_workspace_bytes(T, k, n)
        smoe.smoe_dispatch_tokens(idx, T, k, n, x, _CODE[x.dtype], x.shape[1], offsets, order, place, xs,
                                  _bytes(need, x.device), need)
        ctx.save_for_backward(place)
        ctx.shape = (T, k, x.shape[1])
        ctx.mark_non_differentiable(offsets, place)
        return xs, offsets, place

    @staticmethod
    @once_differentiable
    def backward(ctx, d_xs, _, __):
        place, = ctx.saved_tensors
        T, k, d = ctx.shape
        d_x = torch.empty(T, d, dtype=d_xs.dtype, device=d_xs.device)
        smoe.smoe_dispatch_tokens_backward(d_xs.contiguous(), _CODE[d_xs.dtype], place, T, k, d, d_x)
        return d_x, None, None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ys, place, w):
        ys, place, w = ys.contiguous(), place.contiguous(), w.contiguous()
        T, k = w.shape
        out = torch.empty(T, ys.shape[1], dtype=ys.dtype, device=ys.device)
        smoe.smoe_combine_tokens(ys, _CODE[ys.dtype], place, w, T, k, ys.shape[1], out)
        ctx.save_for_backward(ys, place, w)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, d_out):
        ys, place, w = ctx.saved_tensors
        T, k = w.shape
        d_ys, d_w = torch.empty_like(ys), torch.empty_like(w)
        smoe.smoe_combine_tokens_backward(d_out.contiguous(), ys, _CODE[ys.dtype], place, w, T, k, ys.shape[1], d_ys, d_w)
        return d_ys, None, d_w


def top_k(logits, k):
    """(indices, weights) of each row's k experts, taken and summed in f32;
    differentiable in logits (of any float type)."""
    _check("logits", logits, (None, None), _FLOATS)
    return _TopK.apply(logits.float(), k)


def dispatch(x, idx, n_experts):
    """(rows sorted by expert, offsets, place); differentiable in x (f32 or
    bf16).  idx: integers [tokens, k], no expert where outside [0, n_experts)."""
    _check("x", x, (None, None), tuple(_CODE))
    _check("idx", idx, (x.shape[0], None), _INTS)
    if idx.dtype != torch.int32:  # the library's type; clamped, so that none wraps into another expert
        idx = idx.long().clamp(-1, n_experts).int()
    return _Dispatch.apply(x, idx, n_experts)


def combine(ys, place, w):
    """The experts' rows (f32 or bf16) back in token order, weighted (by any
    float type, in f32); differentiable in both.  place: as dispatch gives it."""
    _check("w", w, (None, None), _FLOATS)
    _check("place", place, (w.numel(),), (torch.int32,))
    _check("ys", ys, (w.numel(), None), tuple(_CODE))
    return _Combine.apply(ys, place, w.float())


def moe_train(x, router, gate_up, down, k):
    """The layer in torch with the routing above, expert by expert (which reads
    the offsets back); every argument may need a gradient.  router [n, d],
    gate_up [n, 2 d_ff, d], down [n, d, d_ff]."""
    n, d_ff = router.shape[0], down.shape[2]
    with torch.autocast(x.device.type, enabled=False):  # the selection is made on f32 logits
        logits = x.float() @ router.float().t()
    idx, w = top_k(logits, k)
    xs, offsets, place = dispatch(x, idx, n)
    ys = []
    at = offsets.tolist()
    for e in range(n):
        h = xs[at[e]:at[e + 1]] @ gate_up[e].t()
        ys.append((torch.nn.functional.silu(h[:, :d_ff]) * h[:, d_ff:]) @ down[e].t())
    ys.append(xs[at[n]:])  # slots without an expert: zeros, not read
    return combine(torch.cat(ys), place, w)


def main():
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev).manual_seed(0)
    n, k, d, d_ff, T = 32, 4, 1024, 512, 48
    router = torch.randn(n, d, generator=g, device=dev) / d ** 0.5
    gate_up = torch.randn(n, 2 * d_ff, d, generator=g, device=dev) / d ** 0.5
    down = torch.randn(n, d, d_ff, generator=g, device=dev) / d_ff ** 0.5
    x = torch.randn(T, d, generator=g, device=dev)
    layer = Q8Layer(router.to(torch.bfloat16).view(torch.int16), gate_up, down, k, T)
    out = layer(x, torch.empty(T, d, dtype=torch.bfloat16, device=dev))
    ref = moe_train(x, router.to(torch.bfloat16).float(), gate_up, down, k)
    print("8-bit layer against the f32 experts: relative difference %.3f" % ((out.float() - ref).norm() / ref.norm()).item())
    params = [p.requires_grad_() for p in (router, gate_up, down)]
    loss = moe_train(x, *params, k).square().mean()
    loss.backward()
    print("loss %.5f, gradient norms %s" % (loss.item(), ["%.4g" % p.grad.norm().item() for p in params]))
    if smoe.smoe_last_device_status() != smoe.SMOE_OK:
        raise RuntimeError("a kernel reported an error")


if __name__ == "__main__":
    main()
