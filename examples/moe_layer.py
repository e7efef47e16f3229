"""A mixture-of-experts layer for a batch of tokens on the many-token calls.

* ``Q8Layer``: serving.  Router, the tokens sorted by expert, gate/up and down
  products with 8-bit weights and activations, the weighted sum back: eight
  calls, nothing read back to the host, so that the whole layer can be
  captured in one CUDA graph.
* ``F8Layer``: the same in 8-bit floating point with a scale for each block of
  128, routed by scores (softmax or sigmoid, with or without a bias and groups).
* ``top_k``, ``route``, ``dispatch``, ``combine``: the same routing under torch's
  autograd (each backward is the library's own call, and has none of its own:
  a second gradient is refused), for training experts written in torch.
* ``experts_f8``: the experts' product in 8-bit floating point under autograd;
  its backward pass is a product with the transposed codes and the weights'
  gradient.  ``moe_train_f8`` trains a whole layer with it, reading nothing back.

``python examples/moe_layer.py`` runs them on a GPU with seeded weights.
"""
import contextlib
import ctypes
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
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}: the calls take the streams of the current device, {torch.cuda.current_device()}")
    if t.dim() != len(shape) or any(w is not None and w != n for n, w in zip(t.shape, shape)):
        raise ValueError(f"{name} has the shape {tuple(t.shape)}, not {shape}")


_FLOATS = (torch.float32, torch.bfloat16, torch.float16, torch.float64)
_INTS = (torch.int32, torch.int64, torch.int16, torch.int8, torch.uint8)


def _adder(t):
    """The node that adds to the leaf t's gradient: one as long as anything holds it."""
    return t.view_as(t).grad_fn.next_functions[0][0]


@contextlib.contextmanager
def _graph_of(*tensors):
    """Around what builds an autograd graph of the tensors.  Torch adds to a leaf's
    gradient on the stream that was current when the leaf's node was made, and ends the
    process where a CUDA graph's capture meets the default stream there.  A capture is
    refused on leaves whose node is held (by an eager graph, whoever built it, or a hook)
    and was made on the default stream, or on one that no backward pass has shown yet."""
    leaves = [t for t in tensors if t.requires_grad and t.is_leaf and t.is_cuda] if torch.is_grad_enabled() else []
    held, key = [], "made on"
    for t in leaves:
        node = _adder(t)
        if key not in node.metadata:
            node.metadata["seen"] = True
            del node  # gone, unless others hold it
            node = _adder(t)
            if not node.metadata.pop("seen", False):
                node.metadata[key] = torch.cuda.current_stream(t.device).cuda_stream
            elif not node.metadata.setdefault("asked", False) and not torch.cuda.is_current_stream_capturing():
                notes, device = node.metadata, t.device
                notes["asked"] = True
                node.register_prehook(lambda _, n=notes, d=device: n.__setitem__(key, torch.cuda.current_stream(d).cuda_stream))
        if not node.metadata.get(key) and torch.cuda.is_current_stream_capturing():
            raise RuntimeError("a captured step needs leaves that no eager graph holds from the default stream (or from one that "
                               "no backward pass has shown): drop that graph, build it on another stream, or detach copies")
        held.append(node)  # until the graph does
    yield


def _bytes(n, device):
    if n == ctypes.c_size_t(-1).value:  # what the library answers to sizes that it refuses
        raise ValueError("no workspace for these sizes: the library refuses them")
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device)


def _logits(x, gate, gate32, logits, stream):
    """logits[t] = gate x[t] in f32: gate bf16, gate32 the same in f32."""
    T, (n, d) = x.shape[0], gate.shape
    if T <= 64 and n % 4 == 0:  # a matvec writes to 16-byte boundaries
        smoe.matvec_bf16_batch([gate] * T, [x.data_ptr() + 4 * d * t for t in range(T)],
                               [logits.data_ptr() + 4 * n * t for t in range(T)], [n] * T, [d] * T, stream)
    else:  # a matvec a token would read the router's weights T times
        with torch.no_grad(), torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext():
            torch.mm(x, gate32.t(), out=logits[:T])


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
        if d % 16 or d_ff % 16:
            raise ValueError(f"d_model {d}, d_ff {d_ff}: both are to be multiples of 16")
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
        _logits(x, self.gate, self.gate32, self.logits, stream)
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


def quantize_weights_f8(w, both=False):
    """e4m3 codes (bytes) and one scale for each 128 x 128 block of w [n, n_out,
    n_in]; both: (codes, scales, and the same of the transposed matrices)."""
    _check("w", w, (None, None, None), tuple(_CODE))
    n, rows, cols = w.shape
    up = lambda m: (m + 127) // 128  # noqa: E731
    u8 = lambda *s: torch.empty(*s, dtype=torch.uint8, device=w.device)  # noqa: E731
    q, scales = u8(n, rows, cols), torch.empty(n, up(rows), up(cols), device=w.device)
    qt, scales_t = (u8(n, cols, rows), torch.empty(n, up(cols), up(rows), device=w.device)) if both else (None, None)
    smoe.smoe_quantize_blocks_f8(w.contiguous(), _CODE[w.dtype], n, rows, cols, q, scales, qt, scales_t)
    return (q, scales, qt, scales_t) if both else (q, scales)


class F8Layer:
    """n_experts experts of d_model -> d_ff -> d_model in 8-bit floating point,
    routed by scores, for up to max_tokens tokens a call.

    gate: router weights bf16 [n_experts, d_model];
    gate_up: [n_experts, 2 d_ff, d_model], the gate rows first, and
    down: [n_experts, d_model, d_ff], f32 or bf16, quantised here;
    bias: f32 [n_experts], added to the scores for the choice, or None;
    score, n_groups, top_groups, group_best, norm, scale: as smoe_route_rows."""

    def __init__(self, gate, gate_up, down, k, max_tokens, bias=None, score=smoe.SMOE_SCORE_SOFTMAX, n_groups=1, top_groups=1,
                 group_best=1, norm=True, scale=1.0):
        n, d, ff = *gate.shape, down.shape[-1]
        _check("gate", gate, (n, d), (torch.bfloat16,))
        _check("gate_up", gate_up, (n, 2 * ff, d), tuple(_CODE))
        _check("down", down, (n, d, ff), tuple(_CODE))
        if d % 16 or ff % 16:
            raise ValueError(f"d_model {d}, d_ff {ff}: both are to be multiples of 16")
        if bias is not None:
            _check("bias", bias, (n,), (torch.float32,))
        dev, self.n, self.d, self.d_ff, self.k, self.max_tokens = gate.device, n, d, ff, k, max_tokens
        self.gate, self.gate32 = gate.contiguous(), gate.float().contiguous()
        self.bias = None if bias is None else bias.contiguous()
        self.choice, self.weighing = (score, n_groups, top_groups, group_best), (int(norm), scale)
        self.gu, self.gu_scales = quantize_weights_f8(gate_up)
        self.dn, self.dn_scales = quantize_weights_f8(down)
        rows = max_tokens * k
        f32 = lambda *s: torch.empty(*s, device=dev)  # noqa: E731
        i32 = lambda *s: torch.empty(*s, dtype=torch.int32, device=dev)  # noqa: E731
        u8 = lambda *s: torch.empty(*s, dtype=torch.uint8, device=dev)  # noqa: E731
        bf = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device=dev)  # noqa: E731
        self.logits, self.idx, self.w = f32(max_tokens, n), i32(max_tokens, k), f32(max_tokens, k)
        self.offsets, self.order, self.place = i32(n + 1), i32(rows), i32(rows)
        self.xq, self.x_scales = u8(max_tokens, d), f32(max_tokens, (d + 127) // 128)
        self.h, self.hq, self.h_scales = bf(rows, 2 * ff), u8(rows, ff), f32(rows, (ff + 127) // 128)
        self.ys = bf(rows, d)
        self.need = max(smoe.smoe_dispatch_workspace_bytes(max_tokens, k, n),
                        smoe.smoe_experts_matmul_f8_workspace_bytes(max_tokens, rows, n, 2 * ff, d),
                        smoe.smoe_experts_matmul_f8_workspace_bytes(rows, rows, n, d, ff))
        self.ws = _bytes(self.need, dev)

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
        R, bf = T * k, smoe.SMOE_BF16
        _logits(x, self.gate, self.gate32, self.logits, stream)
        smoe.smoe_route_rows(self.logits, T, n, n, self.bias, *self.choice, k, *self.weighing, self.idx, self.w, stream)
        smoe.smoe_dispatch_tokens(self.idx, T, k, n, None, smoe.SMOE_F32, 0, self.offsets, self.order, self.place, None,
                                  self.ws, self.need, stream)
        smoe.smoe_quantize_rows_f8(x, smoe.SMOE_F32, smoe.SMOE_Q8_PLAIN, T, d, self.xq, self.x_scales, stream)
        smoe.smoe_experts_matmul_f8(self.xq, self.x_scales, T, self.order, k, self.offsets, R, n, self.gu, self.gu_scales,
                                    2 * ff, d, self.h, bf, self.ws, self.need, stream)
        smoe.smoe_quantize_rows_f8(self.h, bf, smoe.SMOE_Q8_SILU_MUL, R, ff, self.hq, self.h_scales, stream)
        smoe.smoe_experts_matmul_f8(self.hq, self.h_scales, R, None, 1, self.offsets, R, n, self.dn, self.dn_scales, d, ff,
                                    self.ys, bf, self.ws, self.need, stream)
        smoe.smoe_combine_tokens(self.ys, bf, self.place, self.w, T, k, d, out, stream)
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


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, bias, k, score, n_groups, top_groups, group_best, norm, scale):
        logits = logits.contiguous()
        T, n = logits.shape
        idx = torch.empty(T, k, dtype=torch.int32, device=logits.device)
        w = torch.empty(T, k, device=logits.device)
        smoe.smoe_route_rows(logits, T, n, n, bias, score, n_groups, top_groups, group_best, k, norm, scale, idx, w)
        ctx.save_for_backward(logits, idx, w)
        ctx.weighing = score, k, norm, scale
        ctx.mark_non_differentiable(idx)
        return idx, w

    @staticmethod
    @once_differentiable
    def backward(ctx, _, d_w):
        logits, idx, w = ctx.saved_tensors
        T, n = logits.shape
        d = torch.empty(T, n, device=w.device)
        smoe.smoe_route_rows_backward(logits, T, n, n, *ctx.weighing, idx, w, d_w.contiguous(), d)
        return (d,) + (None,) * 8


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


def _product_f8(x, w, w_scales, offsets):
    """Rows x [R, n_in] (sorted by expert), quantised, by codes w [n, n_out, n_in]."""
    (R, n_in), (n, n_out, _) = x.shape, w.shape
    xq = torch.empty(R, n_in, dtype=torch.uint8, device=x.device)
    x_scales = torch.empty(R, (n_in + 127) // 128, device=x.device)
    y = torch.empty(R, n_out, dtype=x.dtype, device=x.device)
    need = smoe.smoe_experts_matmul_f8_workspace_bytes(R, R, n, n_out, n_in)
    smoe.smoe_quantize_rows_f8(x, _CODE[x.dtype], smoe.SMOE_Q8_PLAIN, R, n_in, xq, x_scales)
    smoe.smoe_experts_matmul_f8(xq, x_scales, R, None, 1, offsets, R, n, w, w_scales, n_out, n_in, y, _CODE[x.dtype],
                                _bytes(need, x.device), need)
    return y


class _ExpertsF8(torch.autograd.Function):
    @staticmethod
    def forward(ctx, xs, w, offsets):
        xs, offsets = xs.contiguous(), offsets.contiguous()
        back, grad = ctx.needs_input_grad[:2]
        codes = quantize_weights_f8(w, back)
        ctx.save_for_backward(xs.to(torch.bfloat16) if grad else None, *(codes[2:] if back else (None, None)), offsets)
        ctx.sizes = xs.shape[0], *w.shape, w.dtype
        return _product_f8(xs, *codes[:2], offsets)

    @staticmethod
    @once_differentiable
    def backward(ctx, d_ys):
        xs, qt, scales_t, offsets = ctx.saved_tensors
        R, n, n_out, n_in, w_type = ctx.sizes
        d_xs = d_w = None
        d_ys = d_ys.contiguous()
        if ctx.needs_input_grad[0]:
            d_xs = _product_f8(d_ys, qt, scales_t, offsets)
        if ctx.needs_input_grad[1]:
            d_w = torch.empty(n, n_out, n_in, dtype=w_type, device=d_ys.device)
            smoe.smoe_experts_weight_grad(d_ys.to(torch.bfloat16), xs, offsets, R, n, n_out, n_in, 0, d_w, _CODE[w_type])
        return d_xs, d_w, None


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
    with _graph_of(logits):
        out = _TopK.apply(logits.float(), k)
    return out


def route(logits, k, bias=None, score=smoe.SMOE_SCORE_SOFTMAX, n_groups=1, top_groups=1, group_best=1, norm=True, scale=1.0):
    """(indices, weights) of each row's k experts by their scores, as
    smoe_route_rows takes them; differentiable in logits (of any float type)."""
    _check("logits", logits, (None, None), _FLOATS)
    if bias is not None:
        _check("bias", bias, (logits.shape[1],), (torch.float32,))
        bias = bias.detach().contiguous()
    with _graph_of(logits):
        out = _Route.apply(logits.float(), bias, k, score, n_groups, top_groups, group_best, int(norm), scale)
    return out


def experts_f8(xs, w, offsets):
    """ys[r] = w[e] xs[r] for the rows r of expert e, [offsets[e], offsets[e + 1]),
    both quantised to 8-bit floating point; differentiable in xs [R, n_in] and w
    [n, n_out, n_in] (each f32 or bf16, n_in and n_out multiples of 16), the
    quantisers being passed through as if they were none.  The rows' gradient is
    the product of the quantised output gradients and the transposed codes, the
    weights' that of both operands in bf16."""
    _check("xs", xs, (None, None), tuple(_CODE))
    _check("w", w, (None, None, xs.shape[1]), tuple(_CODE))
    _check("offsets", offsets, (w.shape[0] + 1,), (torch.int32,))
    if w.shape[1] % 16 or w.shape[2] % 16:
        raise ValueError(f"matrices of {tuple(w.shape[1:])}: both sizes are to be multiples of 16")
    with _graph_of(xs, w):
        ys = _ExpertsF8.apply(xs, w, offsets)
    return ys


def dispatch(x, idx, n_experts):
    """(rows sorted by expert, offsets, place); differentiable in x (f32 or
    bf16).  idx: integers [tokens, k], no expert where outside [0, n_experts)."""
    _check("x", x, (None, None), tuple(_CODE))
    _check("idx", idx, (x.shape[0], None), _INTS)
    if idx.dtype != torch.int32:  # the library's type; clamped, so that none wraps into another expert
        idx = idx.long().clamp(-1, n_experts).int()
    with _graph_of(x):
        out = _Dispatch.apply(x, idx, n_experts)
    return out


def combine(ys, place, w):
    """The experts' rows (f32 or bf16) back in token order, weighted (by any
    float type, in f32); differentiable in both.  place: as dispatch gives it."""
    _check("w", w, (None, None), _FLOATS)
    _check("place", place, (w.numel(),), (torch.int32,))
    _check("ys", ys, (w.numel(), None), tuple(_CODE))
    with _graph_of(ys, w):
        out = _Combine.apply(ys, place, w.float())
    return out


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


def moe_train_f8(x, router, gate_up, down, k, bias=None, **how):
    """The layer in 8-bit floating point, routed by scores (how: as route takes
    it); nothing is read back, so that a step can be captured in a CUDA graph.
    x bf16 or f32; every argument but bias may need a gradient.  A capture is refused
    while an eager graph that was built on the default stream holds the same leaves."""
    n, d_ff = router.shape[0], down.shape[2]
    # (the selection is made on f32 logits)
    with _graph_of(x, router, gate_up, down), torch.autocast(x.device.type, enabled=False):
        logits = x.float() @ router.float().t()
        idx, w = route(logits, k, bias, **how)
        xs, offsets, place = dispatch(x, idx, n)
        h = experts_f8(xs, gate_up, offsets)
        ys = experts_f8(torch.nn.functional.silu(h[:, :d_ff]) * h[:, d_ff:], down, offsets)
        out = combine(ys, place, w)
    return out


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
    layer = F8Layer(router.to(torch.bfloat16), gate_up, down, k, T)
    out = layer(x, torch.empty(T, d, dtype=torch.bfloat16, device=dev))
    print("8-bit floating-point layer:              relative difference %.3f" % ((out.float() - ref).norm() / ref.norm()).item())
    for train in (moe_train, moe_train_f8):
        params = [p.detach().clone().requires_grad_() for p in (router, gate_up, down)]
        loss = train(x, *params, k).square().mean()
        loss.backward()
        print("%s: loss %.5f, gradient norms %s" % (train.__name__, loss.item(), ["%.4g" % p.grad.norm().item() for p in params]))
    if smoe.smoe_last_device_status() != smoe.SMOE_OK:
        raise RuntimeError("a kernel reported an error")


if __name__ == "__main__":
    main()
