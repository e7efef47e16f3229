"""Python binding of libsmoe.so (include/smoe.h): group-quantized routed-expert
GEMVs for GB300.

Argument marshalling only: each function below has the name of the C entry
point it calls, turns tensors into device pointers and a stream into a
cudaStream_t, and raises SmoeError when the call returns a non-zero status.
Every step of the computation runs in the library's CUDA kernels; there is no
Python or CPU implementation here and no fallback.  If the library has not
been built, importing this package raises ImportError.

Pointer arguments accept a torch.Tensor (its data_ptr()), an int device
address, or None (NULL).  `stream` accepts a torch.cuda.Stream, an int
cudaStream_t, or None for torch's current stream on the current device.

One MoE layer for one token, every step on the GPU and no host round trip
(the four calls can be captured in one CUDA graph)::

    import moe_expert_ffn_smoe_gb300 as smoe
    # once, when the weights are loaded: device tables of expert pointers
    tabs = [smoe.pointer_table(ts, dev) for ts in (gc, gs, uc, us, dc, ds)]
    # per token; gate: bf16 bits [n_experts, d_model] as int16; x: f32 [d_model]
    smoe.smoe_route_topk_bf16(gate, x, n_experts, d_model, k, logits, idx, w)
    smoe.smoe_experts_ffn_routed_q4(n_experts, k, *tabs, idx, x, expert_out,
                                    d_model, d_ff, group, ws, ws_bytes)
    smoe.smoe_combine(k, expert_out, w, out, d_model)

(`ws`: smoe_experts_ffn_routed_workspace_bytes(k, d_ff) bytes.)  With the
selection on the host, smoe_experts_ffn_q4 takes host lists of the selected
experts' tensors instead.  Several tokens per expert go through
smoe_experts_ffn_batch_q4/q2; a dense bf16 matvec is matvec_bf16, many of
them in one submission matvec_bf16_batch.
"""
import ctypes
import operator
import os
import types

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsmoe.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -c \"import __graft_entry__ as g; g.build()\"` "
        "(the library has no CPU fallback)")

_lib = ctypes.CDLL(LIB_PATH)
try:
    from . import _binding  # noqa: E402  (the same library, arguments marshalled in C)
except ImportError:  # built without Python's headers
    _binding = None
try:
    from . import _binding_f8  # noqa: E402
except ImportError:
    _binding_f8 = None

SMOE_OK = 0
SMOE_ERR_NULL = 1
SMOE_ERR_ALIGN = 2
SMOE_ERR_SHAPE = 3
SMOE_ERR_WORKSPACE = 4
SMOE_ERR_LAUNCH = 5
SMOE_ERR_TIMEOUT = 6
SMOE_ERR_ALIAS = 7
SMOE_ERR_MEMORY = 8
SMOE_ERR_ROUTE = 9
SMOE_MAX_ROUTED_SLOTS = 64
SMOE_MAX_COLS = 32768
SMOE_NOALLOC_SCRATCH_BYTES = 32 << 20
SMOE_FFN_SYNC_BYTES = 512

_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float
_SZ = ctypes.c_size_t

_SIGS = {
    "smoe_abi_version": ([], _I),
    "smoe_status_string": ([_I], ctypes.c_char_p),
    "smoe_gate_up_q4": ([_P, _P, _P, _P, _P, _P, _I, _I, _I, _P], _I),
    "smoe_gate_up_q2": ([_P, _P, _P, _P, _P, _P, _I, _I, _I, _P], _I),
    "smoe_down_q4": ([_P, _P, _P, _P, _I, _I, _I, _P], _I),
    "smoe_down_q2": ([_P, _P, _P, _P, _I, _I, _I, _P], _I),
    "matvec_bf16": ([_P, _P, _P, _I, _I, _P], _I),
    "matvec_bf16_batch": ([_I, _P, _P, _P, _P, _P, _P], _I),
    "smoe_experts_gate_up_q4": ([_I, _P, _P, _P, _P, _P, _P, _I, _I, _I, _P], _I),
    "smoe_experts_gate_up_q2": ([_I, _P, _P, _P, _P, _P, _P, _I, _I, _I, _P], _I),
    "smoe_experts_down_q4": ([_I, _P, _P, _P, _P, _I, _I, _I, _P], _I),
    "smoe_experts_down_q2": ([_I, _P, _P, _P, _P, _I, _I, _I, _P], _I),
    "smoe_experts_ffn_workspace_bytes": ([_I, _I], _SZ),
    "smoe_experts_ffn_q4": ([_I, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _SZ, _P], _I),
    "smoe_experts_ffn_q2": ([_I, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _SZ, _P], _I),
    "smoe_ffn_batch_workspace_bytes": ([_I, _I, _I, _I], _SZ),
    "ffn_batch_q4": ([_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _SZ, _P], _I),
    "ffn_batch_q2": ([_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _SZ, _P], _I),
    "smoe_experts_ffn_routed_workspace_bytes": ([_I, _I], _SZ),
    "smoe_experts_ffn_routed_q4": ([_I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _SZ, _P], _I),
    "smoe_experts_ffn_routed_q2": ([_I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _SZ, _P], _I),
    "smoe_route_topk_bf16": ([_P, _P, _I, _I, _I, _P, _P, _P, _P], _I),
    "smoe_combine": ([_I, _P, _P, _P, _I, _P], _I),
    "smoe_experts_ffn_batch_workspace_bytes": ([_I, _P, _I, _I, _I], _SZ),
    "smoe_experts_ffn_batch_q4": ([_I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _SZ, _P], _I),
    "smoe_experts_ffn_batch_q2": ([_I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _SZ, _P], _I),
    "ffn_batch_q4_noalloc": ([_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P], _I),
    "smoe_topk_rows": ([_P, _I, _I, _I, _I, _P, _P, _P], _I),
    "smoe_topk_rows_backward": ([_P, _P, _P, _I, _I, _I, _P, _P], _I),
    "smoe_dispatch_workspace_bytes": ([_I, _I, _I], _SZ),
    "smoe_dispatch_tokens": ([_P, _I, _I, _I, _P, _I, _I, _P, _P, _P, _P, _P, _SZ, _P], _I),
    "smoe_dispatch_tokens_backward": ([_P, _I, _P, _I, _I, _I, _P, _P], _I),
    "smoe_combine_tokens": ([_P, _I, _P, _P, _I, _I, _I, _P, _P], _I),
    "smoe_combine_tokens_backward": ([_P, _P, _I, _P, _P, _I, _I, _I, _P, _P, _P], _I),
    "smoe_quantize_rows_q8": ([_P, _I, _I, _I, _I, _P, _P, _P], _I),
    "smoe_matmul_q8_workspace_bytes": ([_I, _I, _I], _SZ),
    "smoe_matmul_q8": ([_P, _P, _I, _P, _P, _I, _I, _P, _I, _P, _SZ, _P], _I),
    "smoe_experts_matmul_q8_workspace_bytes": ([_I, _I, _I, _I, _I], _SZ),
    "smoe_experts_matmul_q8": ([_P, _P, _I, _P, _I, _P, _I, _I, _P, _P, _I, _I, _P, _I, _P, _SZ, _P], _I),
    "smoe_route_rows": ([_P, _I, _I, _I, _P, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P], _I),
    "smoe_route_rows_backward": ([_P, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P, _P, _P], _I),
    "smoe_quantize_rows_f8": ([_P, _I, _I, _I, _I, _P, _P, _P], _I),
    "smoe_quantize_blocks_f8": ([_P, _I, _I, _I, _I, _P, _P, _P, _P, _P], _I),
    "smoe_matmul_f8_workspace_bytes": ([_I, _I, _I], _SZ),
    "smoe_matmul_f8": ([_P, _P, _I, _P, _P, _I, _I, _P, _I, _P, _SZ, _P], _I),
    "smoe_experts_matmul_f8_workspace_bytes": ([_I, _I, _I, _I, _I], _SZ),
    "smoe_experts_matmul_f8": ([_P, _P, _I, _P, _I, _P, _I, _I, _P, _P, _I, _I, _P, _I, _P, _SZ, _P], _I),
    "smoe_experts_weight_grad": ([_P, _P, _P, _I, _I, _I, _I, _I, _P, _I, _P], _I),
    "smoe_last_device_status": ([_P], _I),
    "smoe_selftest_bounded_wait": ([_I, _P], _I),
    "smoe_copy": ([_P, _P, ctypes.c_size_t, _P], _I),
}
for _name, (_args, _res) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.argtypes = _args
    _f.restype = _res

EXPORTED = tuple(_SIGS)


class SmoeError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: status {status} ({smoe_status_string(status)})")


def _ptr(a):
    if a is None:
        return None
    if isinstance(a, int):
        return a
    return a.data_ptr()


_current = None  # () -> cudaStream_t of torch's current stream on the current device


def _current_stream():
    """torch's current stream; the lookup is settled by the first call that
    finds a device (asking torch.cuda.is_available() and building a Stream
    object on every call cost as much as a small call's launch)."""
    global _current
    if _current is None:
        import torch
        if not torch.cuda.is_available():
            return None
        torch.cuda.current_stream()  # initialises CUDA
        raw, device = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
        if raw is not None and device is not None:
            _current = lambda: raw(device())  # noqa: E731
        else:
            _current = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
    return _current()


def _stream(s):
    if s is None:
        return _current_stream()
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _by_ctypes(name):
    """_binding's function of that name through ctypes: about 1 us more a call."""
    params, f = _SIGS[name][0][:-1], getattr(_lib, name)

    def integer(a):
        a = operator.index(a)
        if not -1 << 31 <= a < 1 << 31:  # ctypes would cut it
            raise OverflowError("an argument does not fit 32 bits")
        return a

    def real(a):
        if isinstance(a, (str, bytes, bytearray)):  # float would read it
            raise TypeError("an argument is no number")
        return float(a)

    convert = [{_P: _ptr, _I: integer, _F: real, _SZ: operator.index}[t] for t in params]

    def call(*args):
        if len(args) != len(params) + 1:
            raise TypeError(f"{name} takes {len(params) + 1} arguments ({len(args)} given)")
        return f(*[c(a) for c, a in zip(convert, args)], _stream(args[-1]))

    return call


if _binding is not None:
    _binding.set_current_stream(_current_stream)
else:
    _binding = types.SimpleNamespace(**{_name: _by_ctypes(_name) for _name in (
        "smoe_topk_rows", "smoe_topk_rows_backward", "smoe_dispatch_tokens", "smoe_dispatch_tokens_backward",
        "smoe_combine_tokens", "smoe_combine_tokens_backward", "smoe_quantize_rows_q8", "smoe_matmul_q8",
        "smoe_experts_matmul_q8")})
if _binding_f8 is not None:
    _binding_f8.set_current_stream(_current_stream)
else:
    _binding_f8 = types.SimpleNamespace(**{_name: _by_ctypes(_name) for _name in (
        "smoe_route_rows", "smoe_route_rows_backward", "smoe_quantize_rows_f8", "smoe_quantize_blocks_f8",
        "smoe_matmul_f8", "smoe_experts_matmul_f8", "smoe_experts_weight_grad")})


def _check(status, where):
    if status != SMOE_OK:
        raise SmoeError(status, where)


def smoe_abi_version():
    return _lib.smoe_abi_version()


def smoe_status_string(status):
    return _lib.smoe_status_string(int(status)).decode()


def smoe_gate_up_q4(gate_codes, gate_scales, up_codes, up_scales, x, hidden, d_ff, d_model, group,
                    stream=None):
    _check(_lib.smoe_gate_up_q4(_ptr(gate_codes), _ptr(gate_scales), _ptr(up_codes), _ptr(up_scales),
                                _ptr(x), _ptr(hidden), d_ff, d_model, group, _stream(stream)),
           "smoe_gate_up_q4")


def smoe_gate_up_q2(gate_codes, gate_scales, up_codes, up_scales, x, hidden, d_ff, d_model, group,
                    stream=None):
    _check(_lib.smoe_gate_up_q2(_ptr(gate_codes), _ptr(gate_scales), _ptr(up_codes), _ptr(up_scales),
                                _ptr(x), _ptr(hidden), d_ff, d_model, group, _stream(stream)),
           "smoe_gate_up_q2")


def smoe_down_q4(down_codes, down_scales, hidden, out, d_model, d_ff, group, stream=None):
    _check(_lib.smoe_down_q4(_ptr(down_codes), _ptr(down_scales), _ptr(hidden), _ptr(out), d_model,
                             d_ff, group, _stream(stream)), "smoe_down_q4")


def smoe_down_q2(down_codes, down_scales, hidden, out, d_model, d_ff, group, stream=None):
    _check(_lib.smoe_down_q2(_ptr(down_codes), _ptr(down_scales), _ptr(hidden), _ptr(out), d_model,
                             d_ff, group, _stream(stream)), "smoe_down_q2")


def _ptr_array(items):
    """A host array of device pointers (ctypes), kept alive by the caller."""
    arr = (ctypes.c_void_p * max(1, len(items)))()
    for i, t in enumerate(items):
        arr[i] = _ptr(t)
    return arr


def _experts_gate_up(fn, name, gate_codes, gate_scales, up_codes, up_scales, x, hidden, d_ff, d_model,
                     group, stream):
    n = len(gate_codes)
    if not (len(gate_scales) == len(up_codes) == len(up_scales) == n):
        raise ValueError(f"{name}: per-expert lists differ in length")
    arrs = [_ptr_array(a) for a in (gate_codes, gate_scales, up_codes, up_scales)]
    _check(fn(n, *arrs, _ptr(x), _ptr(hidden), d_ff, d_model, group, _stream(stream)), name)


def smoe_experts_gate_up_q4(gate_codes, gate_scales, up_codes, up_scales, x, hidden, d_ff, d_model,
                            group, stream=None):
    """Per-expert lists of tensors; hidden is [n_experts, d_ff]."""
    _experts_gate_up(_lib.smoe_experts_gate_up_q4, "smoe_experts_gate_up_q4", gate_codes, gate_scales,
                     up_codes, up_scales, x, hidden, d_ff, d_model, group, stream)


def smoe_experts_gate_up_q2(gate_codes, gate_scales, up_codes, up_scales, x, hidden, d_ff, d_model,
                            group, stream=None):
    _experts_gate_up(_lib.smoe_experts_gate_up_q2, "smoe_experts_gate_up_q2", gate_codes, gate_scales,
                     up_codes, up_scales, x, hidden, d_ff, d_model, group, stream)


def _experts_down(fn, name, down_codes, down_scales, hidden, out, d_model, d_ff, group, stream):
    n = len(down_codes)
    if len(down_scales) != n:
        raise ValueError(f"{name}: per-expert lists differ in length")
    arrs = [_ptr_array(a) for a in (down_codes, down_scales)]
    _check(fn(n, *arrs, _ptr(hidden), _ptr(out), d_model, d_ff, group, _stream(stream)), name)


def smoe_experts_down_q4(down_codes, down_scales, hidden, out, d_model, d_ff, group, stream=None):
    """Per-expert lists of tensors; hidden [n_experts, d_ff], out [n_experts, d_model]."""
    _experts_down(_lib.smoe_experts_down_q4, "smoe_experts_down_q4", down_codes, down_scales, hidden, out,
                  d_model, d_ff, group, stream)


def smoe_experts_down_q2(down_codes, down_scales, hidden, out, d_model, d_ff, group, stream=None):
    _experts_down(_lib.smoe_experts_down_q2, "smoe_experts_down_q2", down_codes, down_scales, hidden, out,
                  d_model, d_ff, group, stream)


def smoe_experts_ffn_workspace_bytes(n_experts, d_ff):
    return _lib.smoe_experts_ffn_workspace_bytes(n_experts, d_ff)


def _experts_ffn(fn, name, gate_codes, gate_scales, up_codes, up_scales, down_codes, down_scales, x, out,
                 d_model, d_ff, group, workspace, workspace_bytes, stream):
    lists = (gate_codes, gate_scales, up_codes, up_scales, down_codes, down_scales)
    n = len(gate_codes)
    if any(len(a) != n for a in lists):
        raise ValueError(f"{name}: per-expert lists differ in length")
    arrs = [_ptr_array(a) for a in lists]
    _check(fn(n, *arrs, _ptr(x), _ptr(out), d_model, d_ff, group, _ptr(workspace), workspace_bytes,
              _stream(stream)), name)


def smoe_experts_ffn_q4(gate_codes, gate_scales, up_codes, up_scales, down_codes, down_scales, x, out,
                        d_model, d_ff, group, workspace, workspace_bytes, stream=None):
    """Per-expert lists of tensors; out [n_experts, d_model]; workspace of
    smoe_experts_ffn_workspace_bytes(n_experts, d_ff) bytes whose first
    SMOE_FFN_SYNC_BYTES are zero before the first call."""
    _experts_ffn(_lib.smoe_experts_ffn_q4, "smoe_experts_ffn_q4", gate_codes, gate_scales, up_codes, up_scales,
                 down_codes, down_scales, x, out, d_model, d_ff, group, workspace, workspace_bytes, stream)


def smoe_experts_ffn_q2(gate_codes, gate_scales, up_codes, up_scales, down_codes, down_scales, x, out,
                        d_model, d_ff, group, workspace, workspace_bytes, stream=None):
    _experts_ffn(_lib.smoe_experts_ffn_q2, "smoe_experts_ffn_q2", gate_codes, gate_scales, up_codes, up_scales,
                 down_codes, down_scales, x, out, d_model, d_ff, group, workspace, workspace_bytes, stream)


def matvec_bf16(w, x, y, rows, cols, stream=None):
    _check(_lib.matvec_bf16(_ptr(w), _ptr(x), _ptr(y), rows, cols, _stream(stream)), "matvec_bf16")


def matvec_bf16_batch(ws, xs, ys, rows, cols, stream=None):
    """Lists of n tensors (or device addresses) and n sizes; one submission."""
    n = len(ws)
    if not (len(xs) == len(ys) == len(rows) == len(cols) == n):
        raise ValueError("matvec_bf16_batch: lists differ in length")
    arrs = [_ptr_array(a) for a in (ws, xs, ys)]
    r = (ctypes.c_int * max(1, n))(*rows)
    c = (ctypes.c_int * max(1, n))(*cols)
    _check(_lib.matvec_bf16_batch(n, *arrs, r, c, _stream(stream)), "matvec_bf16_batch")


def smoe_ffn_batch_workspace_bytes(T, d_model, d_ff, group):
    return _lib.smoe_ffn_batch_workspace_bytes(T, d_model, d_ff, group)


def ffn_batch_q4(gate_codes, gate_scales, up_codes, up_scales, down_codes, down_scales, X, Y, T,
                 d_model, d_ff, group, workspace, workspace_bytes, stream=None):
    _check(_lib.ffn_batch_q4(_ptr(gate_codes), _ptr(gate_scales), _ptr(up_codes), _ptr(up_scales),
                             _ptr(down_codes), _ptr(down_scales), _ptr(X), _ptr(Y), T, d_model,
                             d_ff, group, _ptr(workspace), workspace_bytes, _stream(stream)),
           "ffn_batch_q4")


def ffn_batch_q2(gate_codes, gate_scales, up_codes, up_scales, down_codes, down_scales, X, Y, T,
                 d_model, d_ff, group, workspace, workspace_bytes, stream=None):
    _check(_lib.ffn_batch_q2(_ptr(gate_codes), _ptr(gate_scales), _ptr(up_codes), _ptr(up_scales),
                             _ptr(down_codes), _ptr(down_scales), _ptr(X), _ptr(Y), T, d_model,
                             d_ff, group, _ptr(workspace), workspace_bytes, _stream(stream)),
           "ffn_batch_q2")


SMOE_MAX_TOP_K = 64
SMOE_MAX_ROUTE_EXPERTS = 8192


def pointer_table(tensors, device):
    """A device array (torch int64 [n]) of the tensors' data pointers: the
    table argument of smoe_experts_ffn_routed_q4/q2, built once."""
    import torch
    return torch.tensor([t.data_ptr() for t in tensors], dtype=torch.int64, device=device)


def smoe_experts_ffn_routed_workspace_bytes(k, d_ff):
    return _lib.smoe_experts_ffn_routed_workspace_bytes(k, d_ff)


def smoe_experts_ffn_routed_q4(n_experts, k, gate_codes, gate_scales, up_codes, up_scales, down_codes,
                               down_scales, top_idx, x, out, d_model, d_ff, group, workspace, workspace_bytes,
                               stream=None):
    """Tables: device arrays of n_experts pointers (pointer_table); top_idx:
    int32 [k] on the device; out [k, d_model]."""
    _check(_lib.smoe_experts_ffn_routed_q4(n_experts, k, _ptr(gate_codes), _ptr(gate_scales), _ptr(up_codes),
                                           _ptr(up_scales), _ptr(down_codes), _ptr(down_scales), _ptr(top_idx),
                                           _ptr(x), _ptr(out), d_model, d_ff, group, _ptr(workspace),
                                           workspace_bytes, _stream(stream)),
           "smoe_experts_ffn_routed_q4")


def smoe_experts_ffn_routed_q2(n_experts, k, gate_codes, gate_scales, up_codes, up_scales, down_codes,
                               down_scales, top_idx, x, out, d_model, d_ff, group, workspace, workspace_bytes,
                               stream=None):
    _check(_lib.smoe_experts_ffn_routed_q2(n_experts, k, _ptr(gate_codes), _ptr(gate_scales), _ptr(up_codes),
                                           _ptr(up_scales), _ptr(down_codes), _ptr(down_scales), _ptr(top_idx),
                                           _ptr(x), _ptr(out), d_model, d_ff, group, _ptr(workspace),
                                           workspace_bytes, _stream(stream)),
           "smoe_experts_ffn_routed_q2")


def smoe_route_topk_bf16(gate_w, x, n_experts, d_model, k, logits, top_idx, top_w, stream=None):
    _check(_lib.smoe_route_topk_bf16(_ptr(gate_w), _ptr(x), n_experts, d_model, k, _ptr(logits), _ptr(top_idx),
                                     _ptr(top_w), _stream(stream)), "smoe_route_topk_bf16")


def smoe_combine(k, expert_out, top_w, out, d_model, stream=None):
    _check(_lib.smoe_combine(k, _ptr(expert_out), _ptr(top_w), _ptr(out), d_model, _stream(stream)),
           "smoe_combine")


def smoe_experts_ffn_batch_workspace_bytes(T, d_model, d_ff, group):
    """T: list of per-expert token counts."""
    t = (ctypes.c_int * max(1, len(T)))(*T)
    return _lib.smoe_experts_ffn_batch_workspace_bytes(len(T), t, d_model, d_ff, group)


def _experts_batch(fn, name, gate_codes, gate_scales, up_codes, up_scales, down_codes, down_scales, X, Y, T,
                   d_model, d_ff, group, workspace, workspace_bytes, stream):
    n = len(T)
    lists = (gate_codes, gate_scales, up_codes, up_scales, down_codes, down_scales, X, Y)
    if any(len(v) != n for v in lists):
        raise ValueError(f"{name}: per-expert lists differ in length")
    arrs = [_ptr_array(v) for v in lists]
    t = (ctypes.c_int * max(1, n))(*T)
    _check(fn(n, *arrs, t, d_model, d_ff, group, _ptr(workspace), workspace_bytes, _stream(stream)), name)


def smoe_experts_ffn_batch_q4(gate_codes, gate_scales, up_codes, up_scales, down_codes, down_scales, X, Y, T,
                              d_model, d_ff, group, workspace, workspace_bytes, stream=None):
    """Per-expert lists of tensors (X[e], Y[e]: [T[e], d_model]) and token counts T."""
    _experts_batch(_lib.smoe_experts_ffn_batch_q4, "smoe_experts_ffn_batch_q4", gate_codes, gate_scales,
                   up_codes, up_scales, down_codes, down_scales, X, Y, T, d_model, d_ff, group, workspace,
                   workspace_bytes, stream)


def smoe_experts_ffn_batch_q2(gate_codes, gate_scales, up_codes, up_scales, down_codes, down_scales, X, Y, T,
                              d_model, d_ff, group, workspace, workspace_bytes, stream=None):
    _experts_batch(_lib.smoe_experts_ffn_batch_q2, "smoe_experts_ffn_batch_q2", gate_codes, gate_scales,
                   up_codes, up_scales, down_codes, down_scales, X, Y, T, d_model, d_ff, group, workspace,
                   workspace_bytes, stream)


def ffn_batch_q4_noalloc(gate_codes, gate_scales, up_codes, up_scales, down_codes, down_scales, X,
                         Y, T, d_model, d_ff, group, stream=None):
    """ffn_batch_q4 with the library's static device workspace, for callers
    that must not allocate device memory (see include/smoe.h)."""
    _check(_lib.ffn_batch_q4_noalloc(_ptr(gate_codes), _ptr(gate_scales), _ptr(up_codes),
                                     _ptr(up_scales), _ptr(down_codes), _ptr(down_scales), _ptr(X),
                                     _ptr(Y), T, d_model, d_ff, group, _stream(stream)),
           "ffn_batch_q4_noalloc")


# ---- many tokens, and experts in 8 bits

SMOE_F32 = 0
SMOE_BF16 = 1
SMOE_MAX_SLOTS = 1 << 30
SMOE_Q8_PLAIN = 0
SMOE_Q8_SILU_MUL = 1


def smoe_topk_rows(logits, n_tokens, n_experts, ld, k, top_idx, top_w, stream=None):
    """The k largest logits of each row (pitch ld floats) and their softmax
    weights; -inf is an expert that is off (index -1, weight 0)."""
    _check(_binding.smoe_topk_rows(logits, n_tokens, n_experts, ld, k, top_idx, top_w,
                                   stream), "smoe_topk_rows")


def smoe_topk_rows_backward(top_idx, top_w, d_top_w, n_tokens, n_experts, k, d_logits, stream=None):
    _check(_binding.smoe_topk_rows_backward(top_idx, top_w, d_top_w, n_tokens, n_experts, k, d_logits,
                                            stream), "smoe_topk_rows_backward")


def smoe_dispatch_workspace_bytes(n_tokens, k, n_experts):
    return _lib.smoe_dispatch_workspace_bytes(n_tokens, k, n_experts)


def smoe_dispatch_tokens(top_idx, n_tokens, k, n_experts, x, dtype, d_model, offsets, order, place, xs,
                         workspace, workspace_bytes, stream=None):
    """Sorts the slots by expert (offsets, order, place) and brings the rows
    of x into that order (x and xs None: the sort alone).  dtype: SMOE_F32 or
    SMOE_BF16, of x and xs."""
    _check(_binding.smoe_dispatch_tokens(top_idx, n_tokens, k, n_experts, x, dtype, d_model, offsets, order,
                                         place, xs, workspace, workspace_bytes,
                                         stream), "smoe_dispatch_tokens")


def smoe_dispatch_tokens_backward(d_xs, dtype, place, n_tokens, k, d_model, d_x, stream=None):
    _check(_binding.smoe_dispatch_tokens_backward(d_xs, dtype, place, n_tokens, k, d_model, d_x,
                                                  stream), "smoe_dispatch_tokens_backward")


def smoe_combine_tokens(ys, dtype, place, top_w, n_tokens, k, d_model, out, stream=None):
    _check(_binding.smoe_combine_tokens(ys, dtype, place, top_w, n_tokens, k, d_model, out,
                                        stream), "smoe_combine_tokens")


def smoe_combine_tokens_backward(d_out, ys, dtype, place, top_w, n_tokens, k, d_model, d_ys, d_top_w,
                                 stream=None):
    _check(_binding.smoe_combine_tokens_backward(d_out, ys, dtype, place, top_w, n_tokens, k, d_model, d_ys,
                                                 d_top_w, stream), "smoe_combine_tokens_backward")


def smoe_quantize_rows_q8(x, dtype, act, rows, cols, q, scales, stream=None):
    """int8 codes and one scale per row of x, or (SMOE_Q8_SILU_MUL) of
    SiLU(gate) * up of rows [gate | up] of 2 cols."""
    _check(_binding.smoe_quantize_rows_q8(x, dtype, act, rows, cols, q, scales,
                                          stream), "smoe_quantize_rows_q8")


def smoe_matmul_q8_workspace_bytes(n_rows, n_out, n_in):
    return _lib.smoe_matmul_q8_workspace_bytes(n_rows, n_out, n_in)


def smoe_matmul_q8(xq, x_scales, n_rows, wq, w_scales, n_out, n_in, y, dtype, workspace, workspace_bytes,
                   stream=None):
    _check(_binding.smoe_matmul_q8(xq, x_scales, n_rows, wq, w_scales, n_out, n_in, y, dtype, workspace,
                                   workspace_bytes, stream), "smoe_matmul_q8")


def smoe_experts_matmul_q8_workspace_bytes(n_src, n_rows, n_experts, n_out, n_in):
    return _lib.smoe_experts_matmul_q8_workspace_bytes(n_src, n_rows, n_experts, n_out, n_in)


def smoe_experts_matmul_q8(xq, x_scales, n_src, order, k, offsets, n_rows, n_experts, wq, w_scales, n_out, n_in,
                           y, dtype, workspace, workspace_bytes, stream=None):
    """order None: xq is already in the sorted order."""
    _check(_binding.smoe_experts_matmul_q8(xq, x_scales, n_src, order, k, offsets, n_rows, n_experts, wq,
                                           w_scales, n_out, n_in, y, dtype, workspace, workspace_bytes,
                                           stream), "smoe_experts_matmul_q8")


# ---- routing by scores, 8-bit floating point, the weights' gradient

SMOE_SCORE_SOFTMAX = 0
SMOE_SCORE_SIGMOID = 1
SMOE_MAX_SCORE_EXPERTS = 1024
SMOE_MAX_GROUPS = 32


def smoe_route_rows(logits, n_tokens, n_experts, ld, bias, score, n_groups, top_groups, group_best, k, norm, scale,
                    top_idx, top_w, stream=None):
    """The k experts of each row by their scores (SMOE_SCORE_SOFTMAX or
    SMOE_SCORE_SIGMOID) plus bias (or None), out of the top_groups best groups,
    and their weights: scale times the scores, over their sum where norm."""
    _check(_binding_f8.smoe_route_rows(logits, n_tokens, n_experts, ld, bias, score, n_groups, top_groups, group_best, k,
                                       norm, scale, top_idx, top_w, stream), "smoe_route_rows")


def smoe_route_rows_backward(logits, n_tokens, n_experts, ld, score, k, norm, scale, top_idx, top_w, d_top_w, d_logits,
                             stream=None):
    _check(_binding_f8.smoe_route_rows_backward(logits, n_tokens, n_experts, ld, score, k, norm, scale, top_idx, top_w,
                                                d_top_w, d_logits, stream), "smoe_route_rows_backward")


def smoe_quantize_rows_f8(x, dtype, act, rows, cols, q, scales, stream=None):
    """e4m3 codes (a byte each) and one scale per row and 128 columns of x, or
    (SMOE_Q8_SILU_MUL) of SiLU(gate) * up of rows [gate | up] of 2 cols."""
    _check(_binding_f8.smoe_quantize_rows_f8(x, dtype, act, rows, cols, q, scales, stream), "smoe_quantize_rows_f8")


def smoe_quantize_blocks_f8(w, dtype, n_mats, rows, cols, q, scales, qt=None, scales_t=None, stream=None):
    """e4m3 codes and one scale per 128 x 128 block of each matrix, and
    (qt, scales_t not None) the same transposed, for the gradient to the rows."""
    _check(_binding_f8.smoe_quantize_blocks_f8(w, dtype, n_mats, rows, cols, q, scales, qt, scales_t, stream),
           "smoe_quantize_blocks_f8")


def smoe_matmul_f8_workspace_bytes(n_rows, n_out, n_in):
    return _lib.smoe_matmul_f8_workspace_bytes(n_rows, n_out, n_in)


def smoe_matmul_f8(xq, x_scales, n_rows, wq, w_scales, n_out, n_in, y, dtype, workspace, workspace_bytes, stream=None):
    _check(_binding_f8.smoe_matmul_f8(xq, x_scales, n_rows, wq, w_scales, n_out, n_in, y, dtype, workspace,
                                      workspace_bytes, stream), "smoe_matmul_f8")


def smoe_experts_matmul_f8_workspace_bytes(n_src, n_rows, n_experts, n_out, n_in):
    return _lib.smoe_experts_matmul_f8_workspace_bytes(n_src, n_rows, n_experts, n_out, n_in)


def smoe_experts_matmul_f8(xq, x_scales, n_src, order, k, offsets, n_rows, n_experts, wq, w_scales, n_out, n_in, y, dtype,
                           workspace, workspace_bytes, stream=None):
    """order None: xq is already in the sorted order."""
    _check(_binding_f8.smoe_experts_matmul_f8(xq, x_scales, n_src, order, k, offsets, n_rows, n_experts, wq, w_scales,
                                              n_out, n_in, y, dtype, workspace, workspace_bytes, stream),
           "smoe_experts_matmul_f8")


def smoe_experts_weight_grad(d_ys, xs, offsets, n_rows, n_experts, n_out, n_in, accumulate, d_w, dtype, stream=None):
    """d_w[e] (of dtype) = the sum over expert e's rows of d_ys[r]^T xs[r] (bf16,
    sorted), or that added to it (accumulate)."""
    _check(_binding_f8.smoe_experts_weight_grad(d_ys, xs, offsets, n_rows, n_experts, n_out, n_in, accumulate, d_w, dtype,
                                                stream), "smoe_experts_weight_grad")


def smoe_last_device_status(stream=None):
    return _lib.smoe_last_device_status(_stream(stream))


def smoe_copy(dst, src, nbytes, stream=None):
    """dst <- src (nbytes) by the SMs; tensors or addresses of device memory or
    pinned host memory."""
    _check(_lib.smoe_copy(_ptr(dst), _ptr(src), nbytes, _stream(stream)), "smoe_copy")


def smoe_selftest_bounded_wait(kind, stream=None):
    """One warp whose bounded wait never succeeds (kind 0: mbarrier, 1: device
    counter); smoe_last_device_status then reports SMOE_ERR_TIMEOUT."""
    _check(_lib.smoe_selftest_bounded_wait(kind, _stream(stream)), "smoe_selftest_bounded_wait")
