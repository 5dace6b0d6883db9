"""Build libvit_b200.so in-tree with nvcc for sm_100a.

    python -m vision_transformer_encoder_fwd_b200.build [--force] [--verbose-ptxas]

The library is two translation units (csrc/vit_api.cu, the encoder, and csrc/ops_api.cu, the
operators; each includes its kernel headers), compiled side by side.  It links the CUDA runtime
statically and resolves the driver's tensor-map encoder at run time, so it needs no libcuda at
link time and cross-compiles on a machine without a GPU.  The objects stay in _build/ and are
kept while none of the files that went into them has changed.
"""
from __future__ import annotations

import argparse
import glob
import os
import shutil
import subprocess
import sys

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
LIB_NAME = "libvit_b200.so"
LIB_PATH = os.path.join(PKG_DIR, LIB_NAME)
OBJ_DIR = os.path.join(PKG_DIR, "_build")
ARCH_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (set NVCC or put CUDA's bin directory on PATH)")


def _sources():
    deps = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
                  glob.glob(os.path.join(ROOT, "include", "*.h")))
    return [os.path.join(CSRC, "vit_api.cu"), os.path.join(CSRC, "ops_api.cu")], deps


def _object_current(obj: str) -> bool:
    """Whether `obj` is newer than every file its dependency list (written by nvcc) names."""
    try:
        with open(obj + ".d") as f:
            names = f.read().replace("\\\n", " ").split(":", 1)[1].split()
        t = os.path.getmtime(obj)
        return all(os.path.getmtime(n) <= t for n in names)
    except (OSError, IndexError):
        return False


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH):
        return False
    t = os.path.getmtime(LIB_PATH)
    return all(os.path.getmtime(d) <= t for d in _sources()[1])


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    if not force and up_to_date():
        return LIB_PATH
    srcs, _ = _sources()
    os.makedirs(OBJ_DIR, exist_ok=True)
    flags = [*ARCH_FLAGS, "-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC,-O2"]
    if verbose_ptxas:
        flags = ["-Xptxas", "-v", *flags]
    objs, running = [], []
    for src in srcs:
        obj = os.path.join(OBJ_DIR, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or verbose_ptxas or not _object_current(obj):
            cmd = [_nvcc(), *flags, "-MMD", "-MF", obj + ".d", "-c", "-o", obj, src]
            running.append(subprocess.Popen(cmd, cwd=ROOT, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True))
    said = [(p.communicate()[0], p.returncode) for p in running]
    tmp = LIB_PATH + ".tmp"
    if all(rc == 0 for _, rc in said):
        p = subprocess.run([_nvcc(), *ARCH_FLAGS, "-shared", "-cudart", "static", "-o", tmp, *objs], cwd=ROOT,
                           capture_output=True, text=True)
        said.append((p.stdout + p.stderr, p.returncode))
    bad = [rc for _, rc in said if rc != 0]
    if bad or verbose_ptxas:
        sys.stderr.write("".join(text for text, _ in said))
    if bad:
        raise RuntimeError(f"nvcc failed with exit code {bad[0]}")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose-ptxas", action="store_true")
    a = ap.parse_args(argv)
    print(build(force=a.force, verbose_ptxas=a.verbose_ptxas))


if __name__ == "__main__":
    main()
