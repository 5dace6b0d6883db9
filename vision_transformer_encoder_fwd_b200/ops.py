"""Operators beside the encoder (the C ABI in include/vit_ops.h): attention over packed sequences,
rotary positions, the root-mean-square norm, 8-bit rows and the linear layer that reads them.

Argument marshalling only, as in the rest of the binding: the work runs in the library's kernels on
the tensors' device, on `stream` or on that device's current stream.  What a call refuses raises
VitError with the library's status.  Outputs that are not given are allocated with torch, on the
stream the call runs on.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
from typing import Optional

from . import VIT_E_INVALID_ARG, VIT_E_SHAPE, VIT_E_UNSUPPORTED, VitError, _check, load_library

ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"plain": 0, "linear": 1, "base": 2, "parts": 3}


class VitRopeTensor(ctypes.Structure):
    _fields_ = [("in_", ctypes.c_void_p), ("out", ctypes.c_void_p), ("in_token", ctypes.c_int64),
                ("in_head", ctypes.c_int64), ("out_token", ctypes.c_int64), ("out_head", ctypes.c_int64),
                ("heads", ctypes.c_int32)]


class VitAttnPacked(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("q_token", ctypes.c_int64), ("q_head", ctypes.c_int64), ("k_token", ctypes.c_int64),
                ("k_head", ctypes.c_int64), ("v_token", ctypes.c_int64), ("v_head", ctypes.c_int64),
                ("out_token", ctypes.c_int64), ("out_head", ctypes.c_int64), ("cu_q", ctypes.c_void_p),
                ("cu_k", ctypes.c_void_p), ("len_k", ctypes.c_void_p), ("Tq", ctypes.c_int64), ("Tk", ctypes.c_int64),
                ("n", ctypes.c_int32), ("heads_q", ctypes.c_int32), ("heads_k", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("type", ctypes.c_int32), ("causal", ctypes.c_int32),
                ("max_q", ctypes.c_int32), ("scale", ctypes.c_float), ("status", ctypes.c_void_p),
                ("wait_ns", ctypes.c_uint64), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


_fns = None
_types = None


def _setup():
    """Signatures of the operator entry points; torch's types by their number in vit_ops.h."""
    global _fns, _types
    import torch
    lib = load_library()
    P, I32, I64, F32, F64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_double
    sigs = {
        "vit_op_rms_norm": [P, I32, I64, P, I64, P, I64, I32, P, I32, F32, I64, I32, P, I32, I64, P, P],
        "vit_op_quant_rows": [P, I32, I64, I64, I32, P, I64, P, P],
        "vit_op_linear_fp8": [P, I64, P, P, I64, P, P, I32, I32, I32, P, I64, P, ctypes.c_uint64, P],
        "vit_op_rope_freqs": [F64, I32, I32, I32, F64, F64, F64, F64, P],
        "vit_op_rope": [ctypes.POINTER(VitRopeTensor), ctypes.POINTER(VitRopeTensor), I32, I64, I32, I32, P, I32, I32, P,
                        I32, F32, I32, P],
        "vit_op_attention_packed_workspace": [ctypes.POINTER(VitAttnPacked), ctypes.POINTER(ctypes.c_size_t)],
        "vit_op_attention_packed": [ctypes.POINTER(VitAttnPacked), P],
        "vit_op_poll": [P],
    }
    fns = {}
    for name, args in sigs.items():
        f = getattr(lib, name)
        f.restype = I32
        f.argtypes = args
        fns[name[len("vit_op_"):]] = f
    _types = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2, torch.float8_e4m3fn: 3}
    _fns = fns


def _fn(name):
    if _fns is None:
        _setup()
    return _fns[name]


def _fail(fn: str, status: int, msg: str):
    raise VitError("vit_op_" + fn, status, msg)


class _Place(contextlib.AbstractContextManager):
    """Where a call runs: its tensors' device, and the stream.  While it is entered that device is
    the current one, and so is the stream (allocations belong to it)."""

    def __init__(self, fn, stream, *tensors):
        import torch
        dev = None
        for t in tensors:
            if t is None:
                continue
            d = t.device
            if d.type != "cuda":
                _fail(fn, VIT_E_INVALID_ARG, "tensors must be on a CUDA device")
            if dev is None:
                dev = d
            elif d != dev:
                _fail(fn, VIT_E_INVALID_ARG, "tensors on different devices")
        self._inner = None
        if stream is not None:
            if stream.device != dev:
                _fail(fn, VIT_E_INVALID_ARG, "the stream is on another device than the tensors")
            self._inner = torch.cuda.stream(stream)
        elif torch.cuda.current_device() != dev.index:
            self._inner = torch.cuda.device(dev)
            stream = torch.cuda.current_stream(dev)
        else:
            stream = torch.cuda.current_stream()
        self.handle = stream.cuda_stream or None

    def __enter__(self):
        if self._inner is not None:
            self._inner.__enter__()
        return self

    def __exit__(self, *exc):
        if self._inner is not None:
            self._inner.__exit__(*exc)
        return False


def _type_of(fn, t):
    if _types is None:
        _setup()
    n = _types.get(t.dtype)
    if n is None:
        _fail(fn, VIT_E_UNSUPPORTED, f"unsupported type {t.dtype}")
    return n


def _rows(fn, t, name):
    """(rows, D, leading dimension) of a matrix with contiguous rows."""
    if t.dim() != 2:
        _fail(fn, VIT_E_SHAPE, f"{name} must be a matrix")
    rows, d = t.shape
    ld, inner = t.stride()
    if inner != 1 and d > 1:
        _fail(fn, VIT_E_INVALID_ARG, f"{name}'s rows must be contiguous")
    return rows, d, (ld if rows > 1 else d)


def _vector(fn, t, name, n, dtype=None):
    if t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        _fail(fn, VIT_E_SHAPE, f"{name} must be a contiguous vector of {n}")
    if dtype is not None and t.dtype != dtype:
        _fail(fn, VIT_E_UNSUPPORTED, f"{name} must be {dtype}")


def rms_norm(x, weight, eps: float = 1e-6, residual=None, residual_out=None, fp8: bool = False, out=None, scales=None,
             stream=None):
    """vit_op_rms_norm: h = x + residual; y = h * weight / sqrt(mean(h^2) + eps) over rows of x [rows, D].

    Returns (out, scales, residual_out): out has x's type, or (fp8, or an 8-bit `out`) is e4m3 with one
    fp32 scale a row, out * scales = y; residual_out holds h in the residual's type (it may be
    `residual` itself) and is None without one."""
    import torch
    fn = "rms_norm"
    with _Place(fn, stream, x, weight, residual, residual_out, out, scales) as at:
        rows, D, ld = _rows(fn, x, "x")
        if out is None:
            out = torch.empty(rows, D, dtype=torch.float8_e4m3fn if fp8 else x.dtype, device=x.device)
        ro, do, ldo = _rows(fn, out, "out")
        e4m3 = out.dtype == torch.float8_e4m3fn
        if fp8 and not e4m3:
            _fail(fn, VIT_E_UNSUPPORTED, "fp8 needs an e4m3 out")
        if e4m3 and scales is None:
            scales = torch.empty(rows, dtype=torch.float32, device=x.device)
        if scales is not None:
            _vector(fn, scales, "scales", rows, torch.float32)
        if (ro, do) != (rows, D):
            _fail(fn, VIT_E_SHAPE, "out must have x's shape")
        _vector(fn, weight, "weight", D)
        r_type, r_ld, h_ld = 0, 0, 0
        if residual is not None:
            if residual_out is None:
                residual_out = torch.empty(rows, D, dtype=residual.dtype, device=x.device)
            if residual.shape != x.shape or residual_out.shape != x.shape or residual_out.dtype != residual.dtype:
                _fail(fn, VIT_E_SHAPE, "residual and residual_out must have x's shape and one type")
            r_type = _type_of(fn, residual)
            r_ld, h_ld = _rows(fn, residual, "residual")[2], _rows(fn, residual_out, "residual_out")[2]
        elif residual_out is not None:
            _fail(fn, VIT_E_INVALID_ARG, "residual_out without residual")
        _check("vit_op_rms_norm", _fn(fn)(
            x.data_ptr(), _type_of(fn, x), ld, None if residual is None else residual.data_ptr(), r_ld,
            None if residual_out is None else residual_out.data_ptr(), h_ld, r_type, weight.data_ptr(),
            _type_of(fn, weight), eps, rows, D, out.data_ptr(), _type_of(fn, out), ldo,
            None if scales is None else scales.data_ptr(), at.handle))
    return out, scales, residual_out


def quant_rows(x, out=None, scales=None, stream=None):
    """vit_op_quant_rows: rows of x in e4m3 with one fp32 scale each; returns (out, scales)."""
    import torch
    fn = "quant_rows"
    with _Place(fn, stream, x, out, scales) as at:
        rows, D, ld = _rows(fn, x, "x")
        if out is None:
            out = torch.empty(rows, D, dtype=torch.float8_e4m3fn, device=x.device)
        if scales is None:
            scales = torch.empty(rows, dtype=torch.float32, device=x.device)
        if out.dtype != torch.float8_e4m3fn:
            _fail(fn, VIT_E_UNSUPPORTED, "out must be e4m3")
        ro, do, ldo = _rows(fn, out, "out")
        if (ro, do) != (rows, D):
            _fail(fn, VIT_E_SHAPE, "out must have x's shape")
        _vector(fn, scales, "scales", rows, torch.float32)
        _check("vit_op_quant_rows", _fn(fn)(x.data_ptr(), _type_of(fn, x), ld, rows, D, out.data_ptr(), ldo,
                                            scales.data_ptr(), at.handle))
    return out, scales


def linear_fp8(a, a_scales, w, w_scales, bias=None, out=None, status=None, stream=None, wait_ns: int = 0):
    """vit_op_linear_fp8: bf16 [M, N] = (a w^T) * a_scales[:, None] * w_scales + bias for e4m3 a [M, K] and
    w [N, K] (nn.Linear layout) as quant_rows and rms_norm(fp8=True) make them; fp32 scales and bias."""
    import torch
    fn = "linear_fp8"
    with _Place(fn, stream, a, a_scales, w, w_scales, bias, out, status) as at:
        M, K, lda = _rows(fn, a, "a")
        N, Kw, ldw = _rows(fn, w, "w")
        if a.dtype != torch.float8_e4m3fn or w.dtype != torch.float8_e4m3fn:
            _fail(fn, VIT_E_UNSUPPORTED, "a and w must be e4m3")
        if K != Kw:
            _fail(fn, VIT_E_SHAPE, "a and w differ in K")
        _vector(fn, a_scales, "a_scales", M, torch.float32)
        _vector(fn, w_scales, "w_scales", N, torch.float32)
        if bias is not None:
            _vector(fn, bias, "bias", N, torch.float32)
        if out is None:
            out = torch.empty(M, N, dtype=torch.bfloat16, device=a.device)
        elif out.dtype != torch.bfloat16:
            _fail(fn, VIT_E_UNSUPPORTED, "out must be bf16")
        mo, no, ldo = _rows(fn, out, "out")
        if (mo, no) != (M, N):
            _fail(fn, VIT_E_SHAPE, "out must be [M, N]")
        if status is not None:
            _vector(fn, status, "status", 1, torch.int32)
        _check("vit_op_linear_fp8", _fn(fn)(
            a.data_ptr(), lda, a_scales.data_ptr(), w.data_ptr(), ldw, w_scales.data_ptr(),
            None if bias is None else bias.data_ptr(), M, N, K, out.data_ptr(), ldo,
            None if status is None else status.data_ptr(), wait_ns, at.handle))
    return out


def rope_freqs(base: float, rotary_dim: int, axes: int = 1, scaling: str = "plain", factor: float = 1.0,
               original_len: float = 0.0, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """vit_op_rope_freqs: CPU float64 tensor of rotary_dim / 2 frequencies (radians per position)."""
    import torch
    fn = "rope_freqs"
    if scaling not in ROPE_SCALINGS:
        _fail(fn, VIT_E_UNSUPPORTED, f"unknown scaling {scaling!r}")
    if rotary_dim < 2 or rotary_dim % 2:
        _fail(fn, VIT_E_SHAPE, "rotary_dim must be even and positive")
    f = torch.empty(rotary_dim // 2, dtype=torch.float64)
    _check("vit_op_rope_freqs", _fn(fn)(base, rotary_dim // 2, axes, ROPE_SCALINGS[scaling], factor, original_len,
                                        beta_fast, beta_slow, f.data_ptr()))
    return f


def _rope_tensor(fn, x, y, T):
    if x.dim() != 3 or y.shape != x.shape or y.dtype != x.dtype or x.shape[0] != T:
        _fail(fn, VIT_E_SHAPE, "q, k and their outputs must be [T, heads, head_dim] of one type")
    (xt, xh, xi), (yt, yh, yi) = x.stride(), y.stride()
    if (xi != 1 or yi != 1) and x.shape[2] > 1:
        _fail(fn, VIT_E_INVALID_ARG, "heads must be contiguous in their last dimension")
    heads = x.shape[1]
    if T == 1:
        xt = yt = 0
    if heads == 1:
        xh = yh = 0
    return VitRopeTensor(x.data_ptr(), y.data_ptr(), xt, xh, yt, yh, heads)


def rope(q, k, positions, freqs, layout: str = "half", gain: float = 1.0, inverse: bool = False, out=None, stream=None):
    """vit_op_rope: rotary positions on q [T, heads, head_dim] and k (or None); returns (q_out, k_out).

    positions: int32 or int64 [T], or [axes, T] for axial positions (the frequencies are then the
    axes' ones one after the other).  freqs: CPU float64 tensor (rope_freqs) of rotary_dim / 2
    values; what a head holds past rotary_dim is copied.  layout: "half" pairs value i with i +
    rotary_dim / 2, "interleaved" 2 i with 2 i + 1.  out: (q_out, k_out), which may be q and k.
    inverse turns back, which is also the gradient's rotation."""
    import torch
    fn = "rope"
    if layout not in ROPE_LAYOUTS:
        _fail(fn, VIT_E_UNSUPPORTED, f"unknown layout {layout!r}")
    q_out, k_out = (None, None) if out is None else out
    with _Place(fn, stream, q, k, positions, q_out, k_out) as at:
        if q.dim() != 3:
            _fail(fn, VIT_E_SHAPE, "q must be [T, heads, head_dim]")
        T, _, d = q.shape
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        if k is None:
            if k_out is not None:
                _fail(fn, VIT_E_INVALID_ARG, "an output for k without k")
        else:
            if k.dtype != q.dtype or k.dim() != 3 or k.shape[2] != d:
                _fail(fn, VIT_E_SHAPE, "k must have q's type and head_dim")
            if k_out is None:
                k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
        if positions.dtype not in (torch.int32, torch.int64):
            _fail(fn, VIT_E_UNSUPPORTED, "positions must be int32 or int64")
        axes = 1 if positions.dim() == 1 else positions.shape[0]
        if positions.dim() not in (1, 2) or positions.shape[-1] != T or not positions.is_contiguous():
            _fail(fn, VIT_E_SHAPE, "positions must be contiguous [T] or [axes, T]")
        if freqs.device.type != "cpu" or freqs.dtype != torch.float64 or freqs.dim() != 1 or not freqs.is_contiguous():
            _fail(fn, VIT_E_INVALID_ARG, "freqs must be a contiguous CPU float64 vector")
        tq = _rope_tensor(fn, q, q_out, T)
        tk = None if k is None else _rope_tensor(fn, k, k_out, T)
        _check("vit_op_rope", _fn(fn)(
            tq, tk, _type_of(fn, q), T, d, 2 * freqs.shape[0], positions.data_ptr(),
            1 if positions.dtype == torch.int64 else 0, axes, freqs.data_ptr(), ROPE_LAYOUTS[layout], gain,
            1 if inverse else 0, at.handle))
    return q_out, k_out


def attention_packed(q, k, v, cu_q, cu_k, len_k=None, causal: bool = False, scale: Optional[float] = None, max_q: int = 0,
                     out=None, status=None, stream=None, wait_ns: int = 0):
    """vit_op_attention_packed: softmax attention of packed sequences, grouped heads; returns out [Tq, heads_q, d].

    q [Tq, heads_q, d], k and v [Tk, heads_k, d], bf16 or fp16, d 64 or 128; any strides but the
    last that are multiples of 8.  Sequence i has query rows cu_q[i] .. cu_q[i+1] - 1 and key rows
    cu_k[i] .. cu_k[i+1] - 1 (int32 [n + 1] on the device), of which the first len_k[i] count if it
    is given (a cache: cu_k holds where each sequence's room begins).  causal: the last query
    sees the last key.  scale: 1 / sqrt(d) by default.  max_q: the longest query length if known
    (it picks kernels, not results).  Rows of out of no sequence are left as they are; an out
    that is allocated here has arbitrary values there."""
    import torch
    fn = "attention_packed"
    with _Place(fn, stream, q, k, v, cu_q, cu_k, len_k, out, status) as at:
        if q.dim() != 3 or k.dim() != 3 or v.shape != k.shape or q.shape[2] != k.shape[2]:
            _fail(fn, VIT_E_SHAPE, "q must be [Tq, heads_q, d], k and v [Tk, heads_k, d]")
        if k.dtype != q.dtype or v.dtype != q.dtype:
            _fail(fn, VIT_E_UNSUPPORTED, "q, k and v must have one type")
        Tq, Hq, d = q.shape
        Tk, Hk, _ = k.shape
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        elif out.shape != q.shape or out.dtype != q.dtype:
            _fail(fn, VIT_E_SHAPE, "out must have q's shape and type")
        n = cu_q.shape[0] - 1 if cu_q.dim() == 1 else -1
        if n < 0:
            _fail(fn, VIT_E_SHAPE, "cu_q must be a vector of n + 1")
        _vector(fn, cu_q, "cu_q", n + 1, torch.int32)
        _vector(fn, cu_k, "cu_k", n + 1, torch.int32)
        if len_k is not None:
            _vector(fn, len_k, "len_k", n, torch.int32)
        if status is not None:
            _vector(fn, status, "status", 1, torch.int32)
        (qt, qh, qi), (kt, kh, ki), (vt, vh, vi), (ot, oh, oi) = q.stride(), k.stride(), v.stride(), out.stride()
        if qi != 1 or ki != 1 or vi != 1 or oi != 1:
            _fail(fn, VIT_E_INVALID_ARG, "heads must be contiguous in their last dimension")
        # the stride of a dimension of one says nothing
        if Tq == 1:
            qt = ot = 0
        if Tk == 1:
            kt = vt = 0
        if Hq == 1:
            qh = oh = 0
        if Hk == 1:
            kh = vh = 0
        args = VitAttnPacked(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), qt, qh, kt, kh, vt, vh, ot, oh, cu_q.data_ptr(),
            cu_k.data_ptr(), None if len_k is None else len_k.data_ptr(), Tq, Tk, n, Hq, Hk, d, _type_of(fn, q),
            1 if causal else 0, max_q, (1.0 / math.sqrt(d) if d else 0.0) if scale is None else scale,
            None if status is None else status.data_ptr(), wait_ns, None, 0)
        need = ctypes.c_size_t()
        _check("vit_op_attention_packed_workspace", _fn("attention_packed_workspace")(args, need))
        if need.value:
            ws = torch.empty(need.value, dtype=torch.uint8, device=q.device)
            args.workspace, args.workspace_bytes = ws.data_ptr(), need.value
        _check("vit_op_attention_packed", _fn(fn)(args, at.handle))
    return out


def op_poll(stream=None) -> None:
    """vit_op_poll: wait for the stream, then raise if an operator's pipeline wait ran out on the
    current device since the last poll (calls that were given no status word of their own)."""
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    with torch.cuda.device(s.device):
        _check("vit_op_poll", _fn("poll")(s.cuda_stream or None))
