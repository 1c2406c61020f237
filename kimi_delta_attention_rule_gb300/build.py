"""Builds libkda.so (the CUDA kernels + C ABI) in-tree for sm_103a, and
_kda_bind.so (the Python side of the attention and cache calls).

Each translation unit is compiled in parallel with nvcc, then linked into
one shared library next to this file; the binding, which alone sees PyTorch's
headers, is one file for the host compiler. Re-running skips an up-to-date build.
Without Python's or PyTorch's headers the library is built all the same, with a
warning; the Python calls that need the binding then raise.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libkda.so")
BIND_SRC = os.path.join(CSRC, "kda_bind.cpp")
BIND = os.path.join(PKG, "_kda_bind.so")
OBJDIR = os.path.join(PKG, "_build")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xptxas", "-v",
              "--expt-relaxed-constexpr", "-I" + INCLUDE, "-I" + CSRC]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in _deps())


def _bind_stamp() -> str:
    return os.path.join(OBJDIR, "bind.txt")


def _bind_against() -> str:
    """What the binding's binary interface goes by; kept beside the objects."""
    import torch
    return "python %s\ntorch %s %s\ncompiler %s\n" % (sys.version, torch.__version__, os.path.dirname(torch.__file__),
                                                     os.environ.get("CXX", "g++"))


def _bind_up_to_date() -> bool:
    if not os.path.exists(BIND) or not os.path.exists(_bind_stamp()):
        return False
    t = os.path.getmtime(BIND)
    if any(os.path.getmtime(p) > t for p in [BIND_SRC] + glob.glob(os.path.join(INCLUDE, "*.h"))):
        return False
    with open(_bind_stamp()) as f:
        return f.read() == _bind_against()


def build_bind(force: bool = False) -> str:
    """The binding module, against the PyTorch that runs this."""
    if not force and _bind_up_to_date():
        return BIND
    try:
        return _compile_bind()
    except Exception:
        if os.path.exists(BIND):  # a stale one: none is better
            os.remove(BIND)
        raise


def _compile_bind() -> str:
    import sysconfig

    import torch
    base = os.path.dirname(torch.__file__)
    inc = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    tmp = BIND + ".tmp%d" % os.getpid()
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-I" + INCLUDE]
    for d in inc:
        cmd += ["-isystem", d]
    cmd += [BIND_SRC, "-o", tmp, "-L" + os.path.join(base, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10",
            "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("%s failed on %s:\n%s\n%s" % (cmd[0], BIND_SRC, r.stdout, r.stderr))
    os.makedirs(OBJDIR, exist_ok=True)
    with open(_bind_stamp(), "w") as f:
        f.write(_bind_against())
    os.replace(tmp, BIND)
    return BIND


def _try_bind(force: bool = False) -> None:
    try:
        build_bind(force)
    except Exception as e:
        warnings.warn("the Python binding of the attention and cache calls is not built: %s" % e)


def build(force: bool = False, verbose: bool = False) -> str:
    """The library (raises if it cannot be built) and, where it can be built, the binding."""
    if not force and up_to_date():
        _try_bind()
        return LIB
    os.makedirs(OBJDIR, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(OBJDIR, os.path.basename(src) + ".o")
        cmd = [cc] + ARCH + NVCC_FLAGS + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed on %s:\n%s\n%s" % (src, r.stdout, r.stderr))
        return obj, r.stderr

    with ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        bind = ex.submit(_try_bind, force)
        results = list(ex.map(compile_one, _sources()))
        bind.result()
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [cc] + ARCH + ["-shared", "-o", tmp] + [o for o, _ in results]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    with open(os.path.join(OBJDIR, "ptxas.log"), "w") as f:
        for _, log in results:
            f.write(log)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
