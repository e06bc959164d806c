"""Build libbsa.so in-tree with nvcc for sm_100a (cross-compiles without a GPU), and _host.so, the
host part of the Python wrappers, with g++.

Usage:  python -m block_sparse_video_bsa_b200.build   (or __graft_entry__.build())
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
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libbsa.so")
HOST = os.path.join(PKG, "_host.so")
BUILD_DIR = os.path.join(PKG, "_build")
HOST_STAMP = os.path.join(BUILD_DIR, "host.built_for")
SOURCES = ["api.cu", "pool_summarize.cu", "select.cu", "attend.cu", "attend_fp8.cu", "quant_fp8.cu",
           "reblock.cu", "extra.cu", "noalloc.cu", "api_block.cu", "rotary.cu", "gate_norm.cu",
           "quant_int8.cu", "linear_int8.cu"]

NVCC_FLAGS = [
    "-O3", "-std=c++17", "-lineinfo",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-Xcompiler", "-fPIC",
    "--expt-relaxed-constexpr",
    "-I", INCLUDE, "-I", CSRC,
]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _newer(target: str, deps) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(d) <= t for d in deps)


def host_built_for() -> str:
    """What _host.so depends on beside its source: it is compiled against torch's and Python's C++ headers."""
    import torch
    return f"torch {torch.__version__}, Python {sys.version_info[0]}.{sys.version_info[1]}"


def _host_command(source: str) -> list:
    import sysconfig

    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    return [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            f'-DBSA_BUILT_FOR="{host_built_for()}"',
            "-I", os.path.join(os.path.dirname(lib), "include"),
            "-I", os.path.join(os.path.dirname(lib), "include", "torch", "csrc", "api", "include"),
            "-I", sysconfig.get_paths()["include"], source,
            "-L", lib, "-lc10", "-ltorch_cpu", "-ltorch_python", "-o", HOST]


def _host_current(source: str) -> bool:
    """_host.so was made from this source, for this torch and Python."""
    try:
        with open(HOST_STAMP) as f:
            return _newer(HOST, [source]) and f.read() == host_built_for()
    except OSError:
        return False


def build(verbose: bool = False, force: bool = False, extra_flags=()) -> str:
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    headers = [os.path.join(CSRC, h) for h in os.listdir(CSRC) if h.endswith((".h", ".cuh"))]
    headers.append(os.path.join(INCLUDE, "bsa.h"))
    objs = []
    jobs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        objs.append(o)
        if force or not _newer(o, [s] + headers):
            jobs.append([nvcc, *NVCC_FLAGS, *extra_flags, "-c", s, "-o", o])

    source = os.path.join(CSRC, "host.cpp")
    host = force or not _host_current(source)
    if host:
        jobs.append(_host_command(source))

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{os.path.basename(cmd[0])} failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)

    with cf.ThreadPoolExecutor(max_workers=len(jobs) or 1) as ex:
        list(ex.map(run, jobs))
    if host:
        with open(HOST_STAMP, "w") as f:
            f.write(host_built_for())
    if force or not _newer(LIB, objs):
        run([nvcc, "-shared", "-gencode", "arch=compute_100a,code=sm_100a", *objs, "-o", LIB])
    return LIB


if __name__ == "__main__":
    build(verbose=True, force="--force" in sys.argv,
          extra_flags=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else [])
    print(LIB)
