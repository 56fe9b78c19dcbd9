"""Build libksa.so (the CUDA library behind include/ksa.h) in-tree for sm_100a, and _marshal.so
(the Python binding's short way to its serving calls, against the installed torch).

Usage: ``python -m block_top_sparse_ksa_b200.build [--force] [--verbose]``.
nvcc cross-compiles without a GPU; the result sits next to this file so it
travels with the source tree.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libksa.so")
MARSHAL = os.path.join(HERE, "_marshal.so")
# ptxas resource report of the last build (registers, spills, shared memory per kernel)
REPORT = os.path.join(HERE, "_build", "ptxas.txt")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is needed to build libksa.so")


def sources():
    return sorted(glob.glob(os.path.join(HERE, "csrc", "*.cu")))


def _inputs():
    return (sources() + glob.glob(os.path.join(HERE, "csrc", "*.cuh")) +
            glob.glob(os.path.join(HERE, "csrc", "*.h")) +
            glob.glob(os.path.join(HERE, "csrc", "*.cpp")) +
            glob.glob(os.path.join(ROOT, "include", "*.h")) + [__file__])


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(MARSHAL):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(MARSHAL))
    return all(os.path.getmtime(p) <= t for p in _inputs())


def _marshal_command():
    import torch
    at = os.path.dirname(torch.__file__)
    include = [os.path.join(ROOT, "include"), os.path.join(at, "include"),
               os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include"),
               sysconfig.get_paths()["include"]]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
            *(f"-I{i}" for i in include), os.path.join(HERE, "csrc", "marshal.cpp"),
            "-o", MARSHAL + ".tmp", f"-L{os.path.join(at, 'lib')}", "-ltorch_python",
            "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date() and os.path.exists(REPORT):
        return LIB
    cmd = [_nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xptxas=-v", "-Xcompiler", "-fPIC",
           "-shared", "-o", LIB + ".tmp", *sources()]
    marshal = _marshal_command()
    beside = subprocess.Popen(marshal, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    said = beside.communicate()[0]
    for code, what, text in ((res.returncode, cmd, res.stdout + res.stderr),
                             (beside.returncode, marshal, said)):
        if code != 0:
            sys.stderr.write(text)
            raise subprocess.CalledProcessError(code, what)
    if verbose:
        sys.stderr.write(res.stderr)
    os.makedirs(os.path.dirname(REPORT), exist_ok=True)
    with open(REPORT, "w") as f:
        f.write(res.stderr)
    os.replace(MARSHAL + ".tmp", MARSHAL)
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="--verbose" in sys.argv)
    print(LIB)
