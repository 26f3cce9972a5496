"""Builds libfa.so (the C-ABI attention library) in-tree with nvcc for sm_103a only.

Each .cu file under csrc/ is compiled to an object in parallel, then linked into
``exact_attention_25_gb300/libfa.so``.  No cmake, no torch extension machinery: the
library is plain C ABI and is loaded with ctypes.  ``build(checked=True)`` makes the
checked variant ``libfa_checked.so`` (-DFA_CHECKED: every direct global access is tested
against its buffer's extent, see fa_checked_build in include/fa.h) from the same sources.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libfa.so")
BUILD_CHECKED = os.path.join(PKG, "_build_checked")
LIB_CHECKED = os.path.join(PKG, "libfa_checked.so")
BINDING = os.path.join(PKG, "_serve.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libfa.so")
    return path


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _headers_mtime() -> float:
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs.append(os.path.join(ROOT, "include", "fa.h"))
    return max(os.path.getmtime(h) for h in hs)


def _compile(src: str, verbose_ptxas: bool, checked: bool = False) -> str:
    obj = os.path.join(BUILD_CHECKED if checked else BUILD, os.path.basename(src)[:-3] + ".o")
    if (os.path.exists(obj) and os.path.getmtime(obj) > os.path.getmtime(src)
            and os.path.getmtime(obj) > _headers_mtime()):
        return obj
    cmd = [nvcc(), *ARCH, *FLAGS, *(["-DFA_CHECKED"] if checked else []), "-c", src,
           "-o", obj + ".tmp"]
    if verbose_ptxas:
        cmd += ["-Xptxas", "-v"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{res.stdout}\n{res.stderr}")
    if verbose_ptxas and res.stderr:
        sys.stderr.write(res.stderr)
    os.replace(obj + ".tmp", obj)
    return obj


def build(force: bool = False, verbose_ptxas: bool = False, checked: bool = False) -> str:
    """Compile every csrc/*.cu for sm_103a and link libfa.so (libfa_checked.so with
    ``checked``); returns its path."""
    bdir, lib = (BUILD_CHECKED, LIB_CHECKED) if checked else (BUILD, LIB)
    os.makedirs(bdir, exist_ok=True)
    if force:
        for f in os.listdir(bdir):
            if not f.endswith(".txt"):  # (the binding's, which is built beside this)
                os.remove(os.path.join(bdir, f))
    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose_ptxas, checked), srcs))
    if (force or not os.path.exists(lib)
            or max(os.path.getmtime(o) for o in objs) > os.path.getmtime(lib)):
        tmp = lib + f".tmp{os.getpid()}"
        cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
        os.replace(tmp, lib)
    return lib


def build_binding(force: bool = False) -> str:
    """Compile the native binding of the serving calls (``_serve.so``, a Python extension that
    allocates through torch and calls the C entry points by address) unless the one that is there was
    built from these sources with this torch and Python; returns its path."""
    import sysconfig

    import torch

    src = os.path.join(CSRC, "serve_binding.cpp")
    header = os.path.join(ROOT, "include", "fa.h")
    made_for = f"torch {torch.__version__} python {sys.version}"
    note = os.path.join(BUILD, "serve_binding.txt")  # what the binding was built for
    if (not force and os.path.exists(BINDING) and _content(note) == made_for
            and os.path.getmtime(BINDING) > max(os.path.getmtime(src), os.path.getmtime(header))):
        return BINDING
    tdir = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-isystem", sysconfig.get_paths()["include"],
           "-isystem", os.path.join(tdir, "include"),
           "-isystem", os.path.join(tdir, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"), src, "-o", tmp,
           "-L", os.path.join(tdir, "lib"), "-Wl,-rpath," + os.path.join(tdir, "lib"),
           "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed for {src}:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, BINDING)
    os.makedirs(BUILD, exist_ok=True)
    with open(note, "w") as f:
        f.write(made_for)
    return BINDING


def _content(path: str) -> str | None:
    if not os.path.exists(path):
        return None
    with open(path) as f:
        return f.read()


def build_all(force: bool = False) -> list[str]:
    """Both variants and the native binding, compiled concurrently."""
    with cf.ThreadPoolExecutor(max_workers=3) as ex:
        jobs = [ex.submit(build, force, checked=c) for c in (False, True)]
        jobs.append(ex.submit(build_binding, force))
        return [j.result() for j in jobs]


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv,
                checked="--checked" in sys.argv))
