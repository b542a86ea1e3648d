"""Compile the CUDA library ``libmxq.so`` for sm_103a, in-tree.

Each ``csrc/*.cu`` is compiled to an object in parallel, then linked into
``affine_bit_matmul_gb300/libmxq.so`` (static CUDA runtime).  ``csrc/torch_calls.cpp``
becomes the Python module ``_calls.so`` beside it, which reads the tensors of the small
calls.  Rebuilds what is older than a source or header of it, and the module also when
Python or torch is another one than it was built for.
"""

from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libmxq.so")
CALLS = os.path.join(PKG, "_calls.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA library cannot be built")
    return path


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def calls_source():
    return os.path.join(CSRC, "torch_calls.cpp")


def _headers():
    return glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(
        os.path.join(INCLUDE, "*.h"))


def _newer(made: str, inputs) -> bool:
    if not os.path.exists(made):
        return False
    t = os.path.getmtime(made)
    return all(os.path.getmtime(p) <= t for p in inputs)


def _versions() -> str:
    """What ``_calls.so`` has to be built for: it loads into this Python and this torch only."""
    import importlib.metadata
    import sys

    try:
        torch = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        import torch as module

        torch = module.__version__
    return "python %s, torch %s\n" % (sys.version, torch)


def _calls_for() -> str:
    """The file that says what ``_calls.so`` was built for."""
    return os.path.join(BUILD, "calls_versions.txt")


def library_up_to_date() -> bool:
    return _newer(LIB, sources() + _headers())


def calls_up_to_date() -> bool:
    if not _newer(CALLS, [calls_source()] + _headers()):
        return False
    try:
        with open(_calls_for()) as f:
            return f.read() == _versions()
    except OSError:
        return False


def up_to_date() -> bool:
    return library_up_to_date() and calls_up_to_date()


def _build_calls(cuda: str):
    import sysconfig

    import torch

    home = os.path.dirname(torch.__file__)
    libs = os.path.join(home, "lib")
    tmp = CALLS + ".tmp%d" % os.getpid()
    cmd = [shutil.which("g++") or "g++", "-O2", "-shared", "-fPIC", "-std=c++17",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI),
           "-I", INCLUDE, "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"),
           "-isystem", os.path.join(home, "include"),
           "-isystem", os.path.join(home, "include", "torch", "csrc", "api", "include"),
           calls_source(), "-o", tmp, "-L", libs, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10",
           "-lc10_cuda", "-Wl,-rpath," + libs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed for %s:\n%s%s" % (calls_source(), r.stdout, r.stderr))
    os.replace(tmp, CALLS)
    with open(_calls_for(), "w") as f:
        f.write(_versions())


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s%s" % (src, r.stdout, r.stderr))
        if verbose:
            print(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        calls = None
        if force or not calls_up_to_date():
            calls = ex.submit(_build_calls, os.path.dirname(os.path.dirname(os.path.realpath(cc))))
        if force or not library_up_to_date():
            objs = list(ex.map(compile_one, sources()))
            tmp = LIB + ".tmp%d" % os.getpid()
            cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"]
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError("link failed:\n%s%s" % (r.stdout, r.stderr))
            os.replace(tmp, LIB)
    # the library does not need torch: it is there also where the module cannot be built
    try:
        if calls is not None:
            calls.result()
    except Exception as e:
        raise RuntimeError("%s is built, but not the module %s: %s" % (LIB, CALLS, e)) from e
    return LIB


if __name__ == "__main__":
    import sys

    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
