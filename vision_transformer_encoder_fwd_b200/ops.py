"""Operators beside the encoder (the C ABI in include/vit_ops.h): attention over packed sequences,
rotary positions, the root-mean-square norm, 8-bit rows and the linear layer that reads them.

Argument marshalling only, as in the rest of the binding, here by an extension module
(csrc/ops_bind.cpp), since a single token's operators take a few microseconds: the work runs in the
library's kernels on the tensors' device, on `stream` or on that device's current stream.  What a
call refuses raises VitError with the library's status.  Outputs that are not given are allocated
with torch, on the stream the call runs on.  Forward only: with grad mode on, a tensor that requires a gradient
is refused.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

from . import VIT_E_SHAPE, VIT_E_UNSUPPORTED, VitError, _build, _check, library_loaded, load_library

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
_bind = None


def _setup():
    """The entry points by their names without vit_op_, with their C signatures."""
    global _fns
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
    _fns = fns


def _fn(name):
    if _fns is None:
        _setup()
    return _fns[name]


def _load():
    """The extension module (built first if it is absent and the compilers are available).

    It is linked against the library by name, so it has to find the very file that this process has loaded or
    will load: with two copies of the library in a process, polls would read the status word of the other one."""
    global _bind
    import torch  # its libraries have to be loaded before the module that uses them
    if not os.path.exists(_build.BIND_PATH):
        before = os.stat(_build.LIB_PATH) if library_loaded() else None
        _build.build()
        if before is not None and not os.path.samestat(before, os.stat(_build.LIB_PATH)):
            raise ImportError("libvit_b200.so was rebuilt, with the operators' binding, after this process had loaded it: "
                              "start the process again")
    load_library()
    from . import _vit_ops
    built = getattr(_vit_ops, "torch_version", "an unknown version")
    if built != torch.__version__:  # it reads tensors by the layout of the headers it was compiled with
        raise ImportError(f"the operators' binding was built against torch {built}, this is {torch.__version__}: "
                          f"run python {_build.__file__}")
    _vit_ops.set_error(VitError)
    _bind = _vit_ops
    return _bind


def _fail(fn: str, status: int, msg: str):
    raise VitError("vit_op_" + fn, status, msg)


def rms_norm(x, weight, eps: float = 1e-6, residual=None, residual_out=None, fp8: bool = False, out=None, scales=None,
             stream=None):
    """vit_op_rms_norm: h = x + residual; y = h * weight / sqrt(mean(h^2) + eps) over rows of x [rows, D].

    Returns (out, scales, residual_out): out has x's type, or (fp8, or an 8-bit `out`) is e4m3 with one
    fp32 scale a row, out * scales = y; residual_out holds h in the residual's type (it may be
    `residual` itself) and is None without one."""
    return (_bind or _load()).rms_norm(x, weight, eps, residual, residual_out, fp8, out, scales, stream)


def quant_rows(x, out=None, scales=None, stream=None):
    """vit_op_quant_rows: rows of x in e4m3 with one fp32 scale each; returns (out, scales)."""
    return (_bind or _load()).quant_rows(x, out, scales, stream)


def linear_fp8(a, a_scales, w, w_scales, bias=None, out=None, status=None, stream=None, wait_ns: int = 0):
    """vit_op_linear_fp8: bf16 [M, N] = (a w^T) * a_scales[:, None] * w_scales + bias for e4m3 a [M, K] and
    w [N, K] (nn.Linear layout) as quant_rows and rms_norm(fp8=True) make them; fp32 scales and bias."""
    return (_bind or _load()).linear_fp8(a, a_scales, w, w_scales, bias, out, status, stream, wait_ns)


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


def rope(q, k, positions, freqs, layout: str = "half", gain: float = 1.0, inverse: bool = False, out=None, stream=None):
    """vit_op_rope: rotary positions on q [T, heads, head_dim] and k (or None); returns (q_out, k_out).

    positions: int32 or int64 [T], or [axes, T] for axial positions (the frequencies are then the
    axes' ones one after the other).  freqs: CPU float64 tensor (rope_freqs) of rotary_dim / 2
    values; what a head holds past rotary_dim is copied.  layout: "half" pairs value i with i +
    rotary_dim / 2, "interleaved" 2 i with 2 i + 1.  out: (q_out, k_out), which may be q and k.
    inverse turns back, which is also the gradient's rotation."""
    code = ROPE_LAYOUTS.get(layout)
    if code is None:
        _fail("rope", VIT_E_UNSUPPORTED, f"unknown layout {layout!r}")
    q_out, k_out = (None, None) if out is None else out
    return (_bind or _load()).rope(q, k, positions, freqs, code, gain, inverse, q_out, k_out, stream)


def attention_packed(q, k, v, cu_q, cu_k, len_k=None, causal: bool = False, scale: Optional[float] = None, max_q: int = 0,
                     out=None, status=None, stream=None, wait_ns: int = 0):
    """vit_op_attention_packed: softmax attention of packed sequences, grouped heads; returns out [Tq, heads_q, d].

    q [Tq, heads_q, d], k and v [Tk, heads_k, d], bf16 or fp16, d 64 or 128; any strides but the
    last that are multiples of 8.  Sequence i has query rows cu_q[i] .. cu_q[i+1] - 1 and key rows
    cu_k[i] .. cu_k[i+1] - 1 (int32 [n + 1] on the device), of which the first len_k[i] count if it
    is given (a cache: cu_k holds where each sequence's room begins).  causal: the last query
    sees the last key.  scale: 1 / sqrt(d) by default.  max_q: the longest query length if known; it
    picks the kernel, and few queries over many keys (new tokens over a cache) are several times slower without
    it.  Any value is right to the precision the header states; the last bits go by the kernel.
    Rows of out of no sequence are left as they are; an out that is allocated here has arbitrary values
    there.  k and v may hold anything outside the sequences' rows; v has to be finite in them, behind the
    causal mask too."""
    return (_bind or _load()).attention_packed(q, k, v, cu_q, cu_k, len_k, causal, scale, max_q, out, status, stream,
                                               wait_ns)


def op_poll(stream=None) -> None:
    """vit_op_poll: wait for the stream, then raise if an operator's pipeline wait ran out on the
    current device since the last poll (calls that were given no status word of their own)."""
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    with torch.cuda.device(s.device):
        _check("vit_op_poll", _fn("poll")(s.cuda_stream or None))
