"""Build libvit_b200.so in-tree with nvcc for sm_100a.

    python -m vision_transformer_encoder_fwd_b200.build [--force] [--verbose-ptxas]

The library is two translation units (csrc/vit_api.cu, the encoder, and csrc/ops_api.cu, the
operators; each includes its kernel headers), compiled side by side.  It links the CUDA runtime
statically and resolves the driver's tensor-map encoder at run time, so it needs no libcuda at
link time and cross-compiles on a machine without a GPU.  The objects stay in _build/ and are
kept while none of the files that went into them has changed.

csrc/ops_bind.cpp becomes _vit_ops.so, the operators' binding: an extension module against torch's
headers that calls the library next to it.
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
ARCH_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (set NVCC or put CUDA's bin directory on PATH)")


def _sources():
    """The library's translation units with their objects."""
    return [(os.path.join(CSRC, n + ".cu"), os.path.join(OBJ_DIR, n + ".o")) for n in ("vit_api", "ops_api")]


def _object_current(obj: str) -> bool:
    """Whether `obj` is newer than every file its dependency list (written by the compiler) names."""
    try:
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
    bind = os.path.join(OBJ_DIR, "ops_bind.o")
    return all(_object_current(o) for o in [*objs, bind]) and _linked(LIB_PATH, objs) and _linked(BIND_PATH, [bind])


def _bind_commands(obj: str):
    """Compile and link commands of the operators' binding."""
    import sysconfig

    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    inc = ["-I" + sysconfig.get_paths()["include"]]
    for d in (os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
              os.path.join(cuda, "include")):
        inc += ["-isystem", d]
    libs = os.path.join(base, "lib")
    cc = os.environ.get("CXX") or "g++"
    abi = f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"
    return ([cc, "-O2", "-fPIC", "-std=c++20", abi, *inc, "-MMD", "-MF", obj + ".d", "-c", "-o", obj,
             os.path.join(CSRC, "ops_bind.cpp")],
            [cc, "-shared", "-o", BIND_PATH + ".tmp", obj, "-L" + libs, "-L" + PKG_DIR, "-ltorch_python", "-ltorch_cpu",
             "-ltorch", "-lc10", "-lc10_cuda", "-l:" + LIB_NAME, "-Wl,-rpath,$ORIGIN"])


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    if not force and up_to_date():
        return LIB_PATH
    os.makedirs(OBJ_DIR, exist_ok=True)
    flags = [*ARCH_FLAGS, "-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC,-O2"]
    if verbose_ptxas:
        flags = ["-Xptxas", "-v", *flags]
    objs, running = [], []
    for src, obj in _sources():
        objs.append(obj)
        if force or verbose_ptxas or not _object_current(obj):
            cmd = [_nvcc(), *flags, "-MMD", "-MF", obj + ".d", "-c", "-o", obj, src]
            running.append(subprocess.Popen(cmd, cwd=ROOT, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True))
    bind = os.path.join(OBJ_DIR, "ops_bind.o")
    bind_compile, bind_link = _bind_commands(bind)
    if force or not _object_current(bind):
        running.append(subprocess.Popen(bind_compile, cwd=ROOT, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True))
    said = [(p.communicate()[0], p.returncode) for p in running]
    # a library that is current stays the file it is: a process may have it loaded
    relink = force or not _linked(LIB_PATH, objs)
    tmp = LIB_PATH + ".tmp"
    if relink and all(rc == 0 for _, rc in said):
        p = subprocess.run([_nvcc(), *ARCH_FLAGS, "-shared", "-cudart", "static", "-o", tmp, *objs], cwd=ROOT,
                           capture_output=True, text=True)
        said.append((p.stdout + p.stderr, p.returncode))
    bad = [rc for _, rc in said if rc != 0]
    if bad or verbose_ptxas:
        sys.stderr.write("".join(text for text, _ in said))
    if bad:
        raise RuntimeError(f"a compiler failed with exit code {bad[0]}")
    if relink:
        os.replace(tmp, LIB_PATH)
    p = subprocess.run(bind_link, cwd=ROOT, capture_output=True, text=True)
    if p.returncode != 0:
        sys.stderr.write(p.stdout + p.stderr)
        raise RuntimeError(f"linking the operators' binding failed with exit code {p.returncode}")
    os.replace(BIND_PATH + ".tmp", BIND_PATH)
    return LIB_PATH


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose-ptxas", action="store_true")
    a = ap.parse_args(argv)
    print(build(force=a.force, verbose_ptxas=a.verbose_ptxas))


if __name__ == "__main__":
    main()
