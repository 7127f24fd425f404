"""Build libtq.so in-tree: every CUDA and C++ source under csrc/, compiled by
nvcc for sm_100a only (no fast-math: the parity contract relies on IEEE
division and square root), linked against the CUDA runtime; and _calls.so, the
Python module over it for the calls of a decode step (csrc/python/, host code).

    python -m kv_cache_vector_15_b200.build [--verbose]
"""

from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libtq.so")
CALLS_SRC = os.path.join(CSRC, "python", "calls.cpp")
CALLS = os.path.join(HERE, "_calls.so")
CALLS_FOR = os.path.join(BUILD, "calls.for")   # the interpreter and the torch that it was built for
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
COMMON = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include"),
          "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _headers_mtime() -> float:
    hs = glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))
    return max((os.path.getmtime(h) for h in hs), default=0.0)


def _compile(src: str, verbose: bool, force: bool = False) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    # objects newer than their source and every header are reused
    if not force and not verbose and os.path.exists(obj) and \
            os.path.getmtime(obj) > max(os.path.getmtime(src), _headers_mtime()):
        return obj
    cmd = [nvcc(), *ARCH, *COMMON, "-c", src, "-o", obj]
    if src.endswith(".cu") and verbose:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    if verbose and r.stderr:
        sys.stderr.write(r.stderr)
    return obj


def build_calls() -> str | None:
    """The Python module: g++ against this interpreter's and torch's headers.
    Without torch there is nothing to build it against, nor a caller of it:
    None, and libtq.so serves its C ABI alone."""
    import sysconfig

    try:
        import torch
    except ImportError:
        return None
    newest = max(os.path.getmtime(CALLS_SRC), os.path.getmtime(os.path.join(ROOT, "include", "tq.h")))
    made_for = f"{sys.version}\n{torch.__version__}\n{os.path.dirname(torch.__file__)}\n"
    try:
        with open(CALLS_FOR) as f:
            same = f.read() == made_for
    except OSError:
        same = False
    if same and os.path.exists(CALLS) and os.path.getmtime(CALLS) > newest:
        return CALLS
    at = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    tmp = CALLS + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", "-w",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", sysconfig.get_paths()["include"], "-isystem", os.path.join(at, "include"), "-isystem",
           os.path.join(at, "include", "torch", "csrc", "api", "include"), "-isystem", os.path.join(cuda, "include"),
           CALLS_SRC, "-o", tmp, "-L", os.path.join(at, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALLS)
    os.makedirs(BUILD, exist_ok=True)
    with open(CALLS_FOR, "w") as f:
        f.write(made_for)
    return CALLS


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 2)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), srcs))
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if build_calls() is None:
        sys.stderr.write("no torch here: _calls.so, which tq.py's paged cache needs, is not built\n")
    return LIB


if __name__ == "__main__":
    print(build(verbose="--verbose" in sys.argv))
