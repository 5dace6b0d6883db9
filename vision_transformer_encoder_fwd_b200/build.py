"""Build libvit_b200.so in-tree with nvcc for sm_100a.

    python -m vision_transformer_encoder_fwd_b200.build [--force] [--verbose-ptxas]

The library is two translation units (csrc/vit_api.cu, the encoder, and csrc/ops_api.cu, the
operators; each includes its kernel headers), compiled side by side.  It links the CUDA runtime
statically and resolves the driver's tensor-map encoder at run time, so it needs no libcuda at
link time and cross-compiles on a machine without a GPU.  The objects stay in _build/ and are
kept while neither the files that went into them nor the compiler's flags have changed.

csrc/ops_bind.cpp becomes _vit_ops.so, the operators' binding: an extension module against torch's
headers that calls the library next to it.  It takes a C++20 compiler and torch; the library needs neither, and
is there without them (for users of the C ABI alone: without torch the binding is left out).
"""
from __future__ import annotations

import argparse
import os
import shutil
import subprocess
import sys

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
LIB_NAME = "libvit_b200.so"
LIB_PATH = os.path.join(PKG_DIR, LIB_NAME)
BIND_PATH = os.path.join(PKG_DIR, "_vit_ops.so")
OBJ_DIR = os.path.join(PKG_DIR, "_build")
BIND_OBJ = os.path.join(OBJ_DIR, "ops_bind.o")
ARCH_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (set NVCC or put CUDA's bin directory on PATH)")


def _sources():
    """The library's translation units with their objects."""
    return [(os.path.join(CSRC, n + ".cu"), os.path.join(OBJ_DIR, n + ".o")) for n in ("vit_api", "ops_api")]


def _object_current(obj: str, how) -> bool:
    """Whether `obj` was compiled with the flags `how` and is newer than every file of this tree that
    its dependency list (written by the compiler) names."""
    try:
        with open(obj + ".flags") as f:
            if f.read() != " ".join(how):
                return False
        with open(obj + ".d") as f:
            names = f.read().replace("\\\n", " ").split(":", 1)[1].split()
        t = os.path.getmtime(obj)
        return all(os.path.getmtime(n) <= t for n in names)
    except (OSError, IndexError):
        return False


def _linked(out: str, objs) -> bool:
    """Whether `out` is there and no older than the objects it is linked from."""
    try:
        return all(os.path.getmtime(o) <= os.path.getmtime(out) for o in objs)
    except OSError:
        return False


def up_to_date() -> bool:
    objs = [obj for _, obj in _sources()]
    if not (all(_object_current(o, _lib_flags()) for o in objs) and _linked(LIB_PATH, objs)):
        return False
    return not _have_torch() or (_object_current(BIND_OBJ, _bind_flags()) and _linked(BIND_PATH, [BIND_OBJ]))


def _have_torch() -> bool:
    try:
        import torch  # noqa: F401
    except ImportError:
        return False
    return True


def _lib_flags():
    return [*ARCH_FLAGS, "-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC,-O2"]


def _bind_flags():
    """Compiler and flags of the operators' binding.  They name what it is compiled against, whose headers its
    dependency list leaves out: torch and its version, its C++ ABI, Python."""
    import sysconfig

    import torch
    base = os.path.join(os.path.dirname(torch.__file__), "include")
    inc = ["-I" + sysconfig.get_paths()["include"]]
    for d in (base, os.path.join(base, "torch", "csrc", "api", "include")):
        inc += ["-isystem", d]
    return [os.environ.get("CXX") or "g++", "-O2", "-fPIC", "-std=c++20",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DVIT_TORCH_VERSION="{torch.__version__}"',
            *inc]


def _bind_link():
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    return [os.environ.get("CXX") or "g++", "-shared", "-o", BIND_PATH + ".tmp", BIND_OBJ, "-L" + libs, "-L" + PKG_DIR,
            "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10", "-lc10_cuda", "-l:" + LIB_NAME, "-Wl,-rpath,$ORIGIN"]


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    if not force and up_to_date():
        return LIB_PATH
    os.makedirs(OBJ_DIR, exist_ok=True)
    running = {}

    def compile_object(src, obj, how, before=(), extra=()):
        if os.path.exists(obj + ".flags"):
            os.remove(obj + ".flags")  # written again once the object is there
        cmd = [*before, *how, *extra, "-MMD", "-MF", obj + ".d", "-c", "-o", obj, src]
        running[obj] = (_start(cmd), how)

    def finish(obj):
        p, how = running.pop(obj, (None, None))
        if p is not None:
            _end(p, verbose_ptxas)
            with open(obj + ".flags", "w") as f:
                f.write(" ".join(how))

    for src, obj in _sources():
        if force or verbose_ptxas or not _object_current(obj, _lib_flags()):
            compile_object(src, obj, _lib_flags(), [_nvcc()], ["-Xptxas", "-v"] if verbose_ptxas else [])
    bind = _have_torch()
    try:
        failed = None
        if bind and (force or not _object_current(BIND_OBJ, _bind_flags())):
            try:
                compile_object(os.path.join(CSRC, "ops_bind.cpp"), BIND_OBJ, _bind_flags(),
                               extra=["-isystem", os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")])
            except OSError as e:  # no such compiler: the library first
                failed = e
        objs = [obj for _, obj in _sources()]
        for obj in objs:
            finish(obj)
        # a library that is current stays the file it is: a process may have it loaded
        if force or not _linked(LIB_PATH, objs):
            _end(_start([_nvcc(), *ARCH_FLAGS, "-shared", "-cudart", "static", "-o", LIB_PATH + ".tmp", *objs]))
            os.replace(LIB_PATH + ".tmp", LIB_PATH)
        if failed is not None:
            raise RuntimeError(f"the operators' binding was not built: {failed}") from failed
        if bind:
            finish(BIND_OBJ)
            _end(_start(_bind_link()))
            os.replace(BIND_PATH + ".tmp", BIND_PATH)
    finally:
        for p, _ in running.values():
            p.communicate()
    return LIB_PATH


def _start(cmd):
    return subprocess.Popen(cmd, cwd=ROOT, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)


def _end(p, show: bool = False) -> None:
    said = p.communicate()[0]
    if show or p.returncode != 0:
        sys.stderr.write(said)
    if p.returncode != 0:
        raise RuntimeError(f"{os.path.basename(p.args[0])} failed with exit code {p.returncode}")


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose-ptxas", action="store_true")
    a = ap.parse_args(argv)
    print(build(force=a.force, verbose_ptxas=a.verbose_ptxas))


if __name__ == "__main__":
    main()
