"""The operator entry points (include/vit_ops.h) without a GPU: every declared function is exported, the
Python structures have the C ones' layout, host validation refuses bad arguments before any CUDA
call, and the frequency helper matches its formulas."""
import ctypes
import math
import os
import re
import subprocess
import tempfile

import pytest
import torch

import vision_transformer_encoder_fwd_b200 as V
from vision_transformer_encoder_fwd_b200 import ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p
A = 1 << 16  # a 16-byte aligned address that no call may touch
BF16, F16, F32, E4M3 = 0, 1, 2, 3


def test_header_and_exports():
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "vit_ops.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(vit_op_\w+)\s*\(", src))
    assert {"vit_op_rms_norm", "vit_op_rope", "vit_op_linear_fp8", "vit_op_attention_packed", "vit_op_poll"} <= names
    V.load_library()
    out = subprocess.run(["nm", "-D", "--defined-only", V.LIB_PATH], capture_output=True, text=True).stdout
    assert names <= set(re.findall(r" T (vit_\w+)", out))
    for n in names:
        assert ops._fn(n[len("vit_op_"):])


def test_struct_layouts_match_c():
    fields = {"vit_rope_tensor": [f if f != "in_" else "in" for f, _ in V.VitRopeTensor._fields_],
              "vit_attn_packed": [f for f, _ in V.VitAttnPacked._fields_]}
    lines = "".join('printf("%%zu ", sizeof(%s));' % s + "".join('printf("%%zu ", offsetof(%s, %s));' % (s, f) for f in fs)
                    for s, fs in fields.items())
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "p.c"), os.path.join(d, "p")
        open(c, "w").write('#include <stdio.h>\n#include <stddef.h>\n#include "vit_ops.h"\nint main(void) {%s return 0;}' % lines)
        subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), c, "-o", exe], check=True)
        got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    want = []
    for s in (V.VitRopeTensor, V.VitAttnPacked):
        want += [ctypes.sizeof(s)] + [getattr(s, f).offset for f, _ in s._fields_]
    assert got == want


def _norm(**kw):
    a = dict(x=A, xt=BF16, xld=64, r=None, rld=0, h=None, hld=0, rt=0, w=A, wt=BF16, eps=1e-6, rows=4, D=64, out=A, ot=BF16,
             old=64, sc=None)
    a.update(kw)
    return ops._fn("rms_norm")(a["x"], a["xt"], a["xld"], a["r"], a["rld"], a["h"], a["hld"], a["rt"], a["w"], a["wt"],
                               a["eps"], a["rows"], a["D"], a["out"], a["ot"], a["old"], a["sc"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(xt=E4M3), V.VIT_E_UNSUPPORTED),
    (dict(xt=7), V.VIT_E_UNSUPPORTED),
    (dict(ot=F16), V.VIT_E_UNSUPPORTED),              # neither x's type nor e4m3
    (dict(wt=F16), V.VIT_E_UNSUPPORTED),
    (dict(r=A, h=A, rt=F16), V.VIT_E_UNSUPPORTED),
    (dict(ot=E4M3), V.VIT_E_INVALID_ARG),              # 8-bit rows without scales
    (dict(sc=A), V.VIT_E_INVALID_ARG),                 # scales without 8-bit rows
    (dict(r=A), V.VIT_E_INVALID_ARG),
    (dict(h=A), V.VIT_E_INVALID_ARG),
    (dict(w=None), V.VIT_E_INVALID_ARG),
    (dict(x=None), V.VIT_E_INVALID_ARG),
    (dict(x=A + 1), V.VIT_E_INVALID_ARG),
    (dict(r=A, h=A + 2, rt=F32, rld=64, hld=64), V.VIT_E_INVALID_ARG),
    (dict(eps=-1.0), V.VIT_E_INVALID_ARG),
    (dict(eps=math.nan), V.VIT_E_INVALID_ARG),
    (dict(eps=math.inf), V.VIT_E_INVALID_ARG),
    (dict(D=0), V.VIT_E_SHAPE),
    (dict(D=32769, xld=32769, old=32769), V.VIT_E_SHAPE),
    (dict(rows=-1), V.VIT_E_SHAPE),
    (dict(xld=-64), V.VIT_E_SHAPE),
    (dict(old=63), V.VIT_E_SHAPE),                     # output rows would overlap
    (dict(r=A, h=A, rld=64, hld=8), V.VIT_E_SHAPE),
    (dict(rows=0), V.VIT_OK),
])
def test_rms_norm_refusals(kw, expect):
    assert _norm(**kw) == expect
    assert V.load_library().vit_last_error() or expect == V.VIT_OK


def test_quant_rows_refusals():
    f = ops._fn("quant_rows")
    assert f(A, E4M3, 64, 4, 64, A, 64, A, None) == V.VIT_E_UNSUPPORTED
    assert f(A, BF16, 64, 4, 64, A, 64, None, None) == V.VIT_E_INVALID_ARG
    assert f(A, BF16, 64, 4, 64, A, 64, A + 2, None) == V.VIT_E_INVALID_ARG
    assert f(A, BF16, 64, 4, 64, A, 32, A, None) == V.VIT_E_SHAPE
    assert f(A, BF16, 64, 0, 64, None, 64, None, None) == V.VIT_OK


def _linear(**kw):
    a = dict(A=A, lda=64, sa=A, W=A, ldw=64, sw=A, b=None, M=4, N=16, K=64, out=A, ldo=16, st=None)
    a.update(kw)
    return ops._fn("linear_fp8")(a["A"], a["lda"], a["sa"], a["W"], a["ldw"], a["sw"], a["b"], a["M"], a["N"], a["K"],
                                 a["out"], a["ldo"], a["st"], 0, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(K=8), V.VIT_E_SHAPE),
    (dict(K=72, lda=80, ldw=80), V.VIT_E_SHAPE),
    (dict(N=12), V.VIT_E_SHAPE),
    (dict(M=-1), V.VIT_E_SHAPE),
    (dict(lda=48), V.VIT_E_SHAPE),
    (dict(lda=72), V.VIT_E_SHAPE),
    (dict(ldw=72), V.VIT_E_SHAPE),
    (dict(ldo=20), V.VIT_E_SHAPE),
    (dict(ldo=8), V.VIT_E_SHAPE),
    (dict(A=A + 8), V.VIT_E_INVALID_ARG),
    (dict(W=A + 8), V.VIT_E_INVALID_ARG),
    (dict(out=A + 8), V.VIT_E_INVALID_ARG),
    (dict(b=A + 4), V.VIT_E_INVALID_ARG),
    (dict(sa=None), V.VIT_E_INVALID_ARG),
    (dict(sw=A + 4), V.VIT_E_INVALID_ARG),
    (dict(st=A + 2), V.VIT_E_INVALID_ARG),
    (dict(M=0), V.VIT_OK),
    (dict(N=0), V.VIT_OK),
])
def test_linear_refusals(kw, expect):
    assert _linear(**kw) == expect


def _rope(T=4, d=64, rd=64, axes=1, layout=0, gain=1.0, type=BF16, pos=A, freqs=None, q=None, qin=A, qout=A, heads=2):
    f = freqs if freqs is not None else (ctypes.c_double * 256)(*([0.5] * 256))
    t = V.VitRopeTensor(qin, qout, heads * d, d, heads * d, d, heads)
    return ops._fn("rope")(ctypes.byref(t), None, type, T, d, rd, pos, 0, axes, f if freqs is not False else None, layout,
                           gain, 0, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(type=E4M3), V.VIT_E_UNSUPPORTED),
    (dict(layout=2), V.VIT_E_UNSUPPORTED),
    (dict(rd=63), V.VIT_E_SHAPE),
    (dict(rd=0), V.VIT_E_SHAPE),
    (dict(rd=66), V.VIT_E_SHAPE),                      # more than the head
    (dict(d=512, rd=258), V.VIT_E_SHAPE),
    (dict(axes=3), V.VIT_E_SHAPE),                     # 32 pairs on three axes
    (dict(axes=5), V.VIT_E_SHAPE),
    (dict(axes=0), V.VIT_E_SHAPE),
    (dict(T=-1), V.VIT_E_SHAPE),
    (dict(heads=-1), V.VIT_E_SHAPE),
    (dict(gain=math.nan), V.VIT_E_INVALID_ARG),
    (dict(freqs=False), V.VIT_E_INVALID_ARG),
    (dict(freqs=(ctypes.c_double * 32)(*([math.inf] * 32))), V.VIT_E_INVALID_ARG),
    (dict(pos=None), V.VIT_E_INVALID_ARG),
    (dict(pos=A + 2), V.VIT_E_INVALID_ARG),
    (dict(qout=None), V.VIT_E_INVALID_ARG),
    (dict(qin=A + 1), V.VIT_E_INVALID_ARG),
    (dict(T=0), V.VIT_OK),
    (dict(heads=0), V.VIT_OK),
])
def test_rope_refusals(kw, expect):
    assert _rope(**kw) == expect


def attn_args(**kw):
    a = dict(q=A, k=A, v=A, out=A, q_token=128, q_head=64, k_token=128, k_head=64, v_token=128, v_head=64, out_token=128,
             out_head=64, cu_q=A, cu_k=A, len_k=None, Tq=8, Tk=8, n=1, heads_q=2, heads_k=2, head_dim=64, type=BF16,
             causal=0, max_q=0, scale=0.125, status=None, wait_ns=0)
    a.update(kw)
    return V.VitAttnPacked(**a)


@pytest.mark.parametrize("kw,expect", [
    (dict(type=F32), V.VIT_E_UNSUPPORTED),
    (dict(head_dim=96), V.VIT_E_UNSUPPORTED),
    (dict(heads_q=3), V.VIT_E_SHAPE),
    (dict(heads_k=0), V.VIT_E_SHAPE),
    (dict(heads_q=65536), V.VIT_E_SHAPE),
    (dict(n=-1), V.VIT_E_SHAPE),
    (dict(Tq=-1), V.VIT_E_SHAPE),
    (dict(Tq=1 << 30), V.VIT_E_SHAPE),
    (dict(Tk=1 << 30), V.VIT_E_SHAPE),
    (dict(k_token=132), V.VIT_E_SHAPE),
    (dict(v_head=-64), V.VIT_E_SHAPE),
    (dict(out_token=1 << 38), V.VIT_E_SHAPE),
    (dict(scale=0.0), V.VIT_E_INVALID_ARG),
    (dict(scale=math.inf), V.VIT_E_INVALID_ARG),
    (dict(scale=math.nan), V.VIT_E_INVALID_ARG),
    (dict(q=None), V.VIT_E_INVALID_ARG),
    (dict(k=None), V.VIT_E_INVALID_ARG),
    (dict(cu_k=None), V.VIT_E_INVALID_ARG),
    (dict(q=A + 8), V.VIT_E_INVALID_ARG),
    (dict(out=A + 8), V.VIT_E_INVALID_ARG),
    (dict(cu_q=A + 2), V.VIT_E_INVALID_ARG),
    (dict(n=0), V.VIT_OK),
    (dict(Tq=0), V.VIT_OK),
])
def test_attention_refusals(kw, expect):
    assert ops._fn("attention_packed")(ctypes.byref(attn_args(**kw)), None) == expect


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(2, 16, dtype=torch.bfloat16)
    with pytest.raises(V.VitError) as e:
        V.rms_norm(x, x[0])
    assert e.value.status == V.VIT_E_INVALID_ARG
    with pytest.raises(V.VitError):
        V.quant_rows(x)


def test_rope_frequencies():
    """base^(-i/p), and its stretched forms, to the last few bits of a double."""
    base, p, factor = 10000.0, 32, 8.0
    plain = [base ** (-i / p) for i in range(p)]

    def close(f, want):
        assert f.dtype == torch.float64 and f.shape == (len(want),)
        assert all(abs(a - b) <= 1e-14 * b for a, b in zip(f.tolist(), want))
    close(V.rope_freqs(base, 2 * p), plain)
    close(V.rope_freqs(base, 2 * p, scaling="linear", factor=factor), [f / factor for f in plain])
    b2 = base * factor ** (p / (p - 1))
    close(V.rope_freqs(base, 2 * p, scaling="base", factor=factor), [b2 ** (-i / p) for i in range(p)])
    parts = []
    for f in plain:
        keep = min(1.0, max(0.0, (f * 4096 / (2 * math.pi) - 1.0) / 31.0))
        parts.append(f / factor * (1 - keep) + f * keep)
    close(V.rope_freqs(base, 2 * p, scaling="parts", factor=factor, original_len=4096), parts)
    half = [base ** (-i / (p // 2)) for i in range(p // 2)]
    close(V.rope_freqs(base, 2 * p, axes=2), half + half)


@pytest.mark.parametrize("kw,expect", [
    (dict(base=0.0), V.VIT_E_INVALID_ARG),
    (dict(base=math.nan), V.VIT_E_INVALID_ARG),
    (dict(rotary_dim=258), V.VIT_E_SHAPE),
    (dict(rotary_dim=7), V.VIT_E_SHAPE),
    (dict(axes=3), V.VIT_E_SHAPE),
    (dict(scaling="linear", factor=0.0), V.VIT_E_INVALID_ARG),
    (dict(scaling="parts", factor=2.0), V.VIT_E_INVALID_ARG),                     # no original length
    (dict(scaling="parts", factor=2.0, original_len=64, beta_fast=1.0, beta_slow=1.0), V.VIT_E_INVALID_ARG),
    (dict(scaling="base", factor=2.0, rotary_dim=2), V.VIT_E_SHAPE),
    (dict(scaling="other"), V.VIT_E_UNSUPPORTED),
])
def test_rope_frequency_refusals(kw, expect):
    a = dict(base=10000.0, rotary_dim=64)
    a.update(kw)
    with pytest.raises(V.VitError) as e:
        V.rope_freqs(**a)
    assert e.value.status == expect


@pytest.mark.parametrize("kw", [dict(workspace=None, workspace_bytes=1 << 30), dict(workspace=A, workspace_bytes=64),
                                dict(workspace=A + 8, workspace_bytes=1 << 30)])
def test_attention_workspace_refusals(kw):
    """Few query rows over long key rows take a workspace: refused where it is missing, too small or misaligned."""
    assert ops._fn("attention_packed")(ctypes.byref(attn_args(max_q=1, Tk=4096, **kw)), None) == V.VIT_E_WORKSPACE


def test_attention_workspace_size():
    need = ctypes.c_size_t(7)
    f = ops._fn("attention_packed_workspace")
    assert f(ctypes.byref(attn_args(max_q=0)), need) == V.VIT_OK and need.value == 0
    assert f(ctypes.byref(attn_args(max_q=1)), need) == V.VIT_OK and need.value == 0
    assert f(ctypes.byref(attn_args(max_q=1, Tk=4096)), need) == V.VIT_OK and 0 < need.value <= 10 << 20
    assert f(ctypes.byref(attn_args(max_q=1, Tk=4096, head_dim=128)), need) == V.VIT_OK and 0 < need.value <= 10 << 20
    assert f(ctypes.byref(attn_args(max_q=1, head_dim=80)), need) == V.VIT_E_UNSUPPORTED
    assert f(ctypes.byref(attn_args(max_q=1)), None) == V.VIT_E_INVALID_ARG


def _copy_of_the_package(to):
    """The package with its headers and built files (times kept, so that nothing in them is stale)."""
    import shutil
    name = os.path.basename(os.path.dirname(V.__file__))
    ops._build.build()
    for d in (name, "include"):
        shutil.copytree(os.path.join(ROOT, d), to / d, ignore=shutil.ignore_patterns("__pycache__"))
    return to / name


def _python(code, cwd, **env):
    import sys
    return subprocess.run([sys.executable, "-c", code], cwd=cwd, capture_output=True, text=True, timeout=600,
                          env={**os.environ, "PYTHONPATH": str(cwd), **env})


def test_binding_built_late_uses_the_loaded_library(tmp_path):
    """A process that has loaded the library and then builds the missing binding has one copy of the library; one
    whose library had to be rebuilt for it is told so."""
    pkg = _copy_of_the_package(tmp_path)
    code = f"""
import os, {pkg.name} as V
V.load_library()
os.remove(V.ops._build.BIND_PATH)
CHANGE
V.ops._load()
files = {{l.split()[4] for l in open("/proc/self/maps") if "libvit_b200.so" in l}}
assert len(files) == 1, files
print("one library")
"""
    res = _python(code.replace("CHANGE", ""), tmp_path)
    assert "one library" in res.stdout, res.stderr[-2000:]
    res = _python(code.replace("CHANGE", "os.utime(V.ops._build._sources()[0][1])"), tmp_path)
    assert res.returncode != 0 and "start the process again" in res.stderr, res.stderr[-2000:]


def test_binding_follows_torch(monkeypatch):
    """A binding of another torch (or of other flags) is stale for the build, and refused when it is loaded."""
    ops._build.build()
    assert ops._build.up_to_date()
    if ops._bind is None:
        ops._load()
    loaded = ops._bind
    with monkeypatch.context() as m:
        m.setenv("CXX", "another-compiler")
        assert not ops._build.up_to_date()
    with monkeypatch.context() as m:
        m.setattr(ops._build, "ARCH_FLAGS", [*ops._build.ARCH_FLAGS, "-G"])
        assert not ops._build.up_to_date()
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "1.0.0")
        assert not ops._build.up_to_date()
        with pytest.raises(ImportError, match="built against torch"):
            ops._load()
    assert ops._build.up_to_date() and ops._load() is loaded


def test_library_builds_without_torch_and_without_a_host_compiler_for_the_binding(tmp_path):
    """nvcc alone is enough for the C ABI."""
    pkg = _copy_of_the_package(tmp_path)
    (pkg / V.ops._build.LIB_NAME).unlink()
    (pkg / "_vit_ops.so").unlink()
    code = f"""
import ctypes, os, runpy, sys
sys.modules["torch"] = None  # importing it raises ImportError
build = runpy.run_path(os.path.join({pkg.name!r}, "build.py"))
assert not build["up_to_date"]()
lib = ctypes.CDLL(build["build"]())
assert lib.vit_op_quant_rows and not os.path.exists(build["BIND_PATH"]) and build["up_to_date"]()
print("C ABI")
"""
    res = _python(code, tmp_path)
    assert "C ABI" in res.stdout, res.stderr[-2000:]
    (pkg / V.ops._build.LIB_NAME).unlink()
    for cxx in ("false", "no-such-compiler"):
        code = f"import runpy; print(runpy.run_path('{pkg.name}/build.py')['build']())"
        res = _python(code, tmp_path, CXX=cxx)
        assert res.returncode != 0 and "RuntimeError" in res.stderr, res.stderr[-2000:]
        assert (pkg / V.ops._build.LIB_NAME).exists() and not (pkg / "_vit_ops.so").exists()


@pytest.mark.parametrize("kw", [
    dict(ot=E4M3, sc=A),                               # 8-bit rows packed at the start of x's memory
    dict(ot=E4M3, sc=A, xt=F32, wt=F32, old=128),
    dict(xld=128),                                     # rows brought together in place
    dict(r=2 * A, h=2 * A, rt=F32, rld=64, hld=128),
    dict(xld=0),                                       # a broadcast row
])
def test_rms_norm_refuses_an_output_on_other_rows(kw):
    """out on x, or residual_out on residual, where row i is not on row i: what a block writes, others still read."""
    assert _norm(**kw) == V.VIT_E_SHAPE


def test_quant_rows_refuses_an_output_on_other_rows():
    f = ops._fn("quant_rows")
    assert f(A, BF16, 64, 4, 64, A, 64, 2 * A, None) == V.VIT_E_SHAPE
    assert f(A, F32, 64, 4, 64, A, 128, 2 * A, None) == V.VIT_E_SHAPE


@pytest.mark.parametrize("kw", [
    dict(out_token=0), dict(out_head=0), dict(out_token=64), dict(out_head=32), dict(out_head=128),
    dict(out_head=8 * 64, out_token=56),
    dict(heads_q=3, heads_k=1, Tq=3, out_head=192, out_token=192),  # interleaved, a token on a head
    dict(heads_q=3, heads_k=1, Tq=4, out_head=192, out_token=136),  # 2 * 192 and 3 * 136 are 24 values apart
])
def test_attention_refuses_an_output_that_overlaps_itself(kw):
    assert ops._fn("attention_packed")(ctypes.byref(attn_args(**{"heads_q": 2, "heads_k": 2, **kw})), None) == V.VIT_E_SHAPE


def test_overlap_rule_against_all_pairs():
    """What attention and rope refuse as an overlapping output, against every pair of heads, for layouts with heads in
    tokens, tokens in heads and interleaved.  No call gets past its checks: the positions (or cu_q) are missing."""
    f = (ctypes.c_double * 32)(*([0.5] * 32))
    seen = set()
    for T in (1, 2, 3, 5):
        for H in (1, 2, 3, 4):
            for st in (0, 1, 3, 4, 6, 8, 9, 12, 17, 20):
                for sh in (0, 2, 4, 5, 8, 10, 12, 16, 23):
                    at = [t * st + h * sh for t in range(T) for h in range(H)]
                    over = any(abs(a - b) < 4 for i, a in enumerate(at) for b in at[:i])
                    seen.add(over)
                    x = V.VitRopeTensor(A, 2 * A, H * 4, 4, st, sh, H)
                    got = ops._fn("rope")(ctypes.byref(x), None, BF16, T, 4, 4, None, 0, 1, f, 0, 1.0, 0, None)
                    assert got == (V.VIT_E_SHAPE if over else V.VIT_E_INVALID_ARG), (T, H, st, sh)
    assert seen == {True, False}


def test_rope_refuses_an_output_on_other_heads():
    f = (ctypes.c_double * 32)(*([0.5] * 32))

    def call(T, heads, in_token, in_head, out_token, out_head):
        x = V.VitRopeTensor(A, A, in_token, in_head, out_token, out_head, heads)
        return ops._fn("rope")(ctypes.byref(x), None, BF16, T, 64, 64, None, 0, 1, f, 0, 1.0, 0, None)
    assert call(4, 2, 256, 64, 128, 64) == V.VIT_E_SHAPE      # brought together in place
    assert call(4, 2, 128, 64, 64, 256) == V.VIT_E_SHAPE      # transposed in place
    assert call(4, 2, 0, 64, 128, 64) == V.VIT_E_SHAPE
    assert call(4, 2, 256, 64, 256, 64) == V.VIT_E_INVALID_ARG  # positions missing: nothing else is wrong
    assert call(1, 2, 7, 64, 9, 64) == V.VIT_E_INVALID_ARG


def test_binding_refuses_what_autograd_would_record():
    """The operators are forward only: with grad mode on, a tensor that requires a gradient is refused, and without it
    the call gets on (here to the check of the device)."""
    bf = torch.bfloat16
    x, w = torch.zeros(2, 16, dtype=bf), torch.ones(16)
    heads, cu = torch.zeros(2, 1, 64, dtype=bf), torch.zeros(2, dtype=torch.int32)
    q8, s8 = torch.zeros(8, 16).to(torch.float8_e4m3fn), torch.ones(8)
    pos, f = torch.zeros(2, dtype=torch.int32), V.rope_freqs(100.0, 64)
    calls = [
        (lambda t: V.rms_norm(t, w), x), (lambda t: V.rms_norm(x, t), w), (lambda t: V.rms_norm(x, w, residual=t), x),
        (lambda t: V.rms_norm(x, w, out=t), x), (lambda t: V.quant_rows(t), x),
        (lambda t: V.linear_fp8(q8, t, q8, s8), s8), (lambda t: V.linear_fp8(q8, s8, q8, s8, bias=t), s8),
        (lambda t: V.rope(t, None, pos, f), heads), (lambda t: V.rope(heads, t, pos, f), heads),
        (lambda t: V.rope(heads, None, pos, t), f),
        (lambda t: V.attention_packed(t, heads, heads, cu, cu), heads), (lambda t: V.attention_packed(heads, heads, t, cu, cu), heads),
    ]
    for call, t in calls:
        leaf = t.clone().requires_grad_()
        for needs in (leaf, leaf * 1):
            with pytest.raises(V.VitError) as e:
                call(needs)
            assert e.value.status == V.VIT_E_UNSUPPORTED and "gradient" in str(e.value)
        for context in (torch.no_grad(), torch.inference_mode()):
            with context, pytest.raises(V.VitError) as e:
                call(leaf)
            assert e.value.status == V.VIT_E_INVALID_ARG
        with pytest.raises(V.VitError) as e:
            call(leaf.detach())
        assert e.value.status == V.VIT_E_INVALID_ARG


def test_binding_refuses_a_negative_wait():
    """As an unsigned limit it would be centuries: no wait is without a bound."""
    q8, s8 = torch.zeros(8, 16).to(torch.float8_e4m3fn), torch.ones(8)
    heads, cu = torch.zeros(2, 1, 64, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: V.linear_fp8(q8, s8, q8, s8, wait_ns=-1),
                 lambda: V.attention_packed(heads, heads, heads, cu, cu, wait_ns=-1)):
        with pytest.raises(V.VitError, match="wait_ns") as e:
            call()
        assert e.value.status == V.VIT_E_INVALID_ARG


def test_binding_that_does_not_name_its_torch_is_refused(monkeypatch):
    """A module of an older checkout."""
    if ops._bind is None:
        ops._load()
    with monkeypatch.context() as m:
        m.delattr(ops._bind, "torch_version")
        with pytest.raises(ImportError, match="built against torch an unknown version"):
            ops._load()
    ops._load()
