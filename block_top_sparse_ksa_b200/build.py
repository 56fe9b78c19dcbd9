"""Build libksa.so (the CUDA library behind include/ksa.h) in-tree for sm_100a, and _marshal.so
(the Python binding's short way to its serving calls, against the installed torch; the binding
does without where it cannot be built).

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

from . import _built_for as built_for

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


def _newer_than_inputs(path: str) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(p) <= os.path.getmtime(path)
                                        for p in _inputs())


def _marshal_up_to_date() -> bool:
    if not _newer_than_inputs(MARSHAL):
        return False
    with open(MARSHAL, "rb") as f:  # it reads tensors by the layout of the torch it was built for
        return built_for().encode() in f.read()


def up_to_date() -> bool:
    return _newer_than_inputs(LIB) and os.path.exists(REPORT) and _marshal_up_to_date()


def _lib_command():
    return [_nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xptxas=-v", "-Xcompiler", "-fPIC",
            "-shared", "-o", LIB + ".tmp", *sources()]


def _marshal_command():
    import torch
    at = os.path.dirname(torch.__file__)
    include = [os.path.join(ROOT, "include"), os.path.join(at, "include"),
               os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include"),
               sysconfig.get_paths()["include"]]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
            f'-DKSA_BUILT_FOR="{built_for()}"',
            *(f"-I{i}" for i in include), os.path.join(HERE, "csrc", "marshal.cpp"),
            "-o", MARSHAL + ".tmp", f"-L{os.path.join(at, 'lib')}", "-ltorch_python",
            "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def _start_marshal():
    """The compiler of _marshal.so, or None and what went wrong."""
    try:
        return subprocess.Popen(_marshal_command(), stdout=subprocess.PIPE,
                                stderr=subprocess.STDOUT, text=True), ""
    except Exception as e:  # no g++, no torch headers: the binding does without
        return None, f"{type(e).__name__}: {e}\n"


def _finish_marshal(beside, said: str) -> None:
    if beside is not None:
        said = beside.communicate()[0]
        if beside.returncode == 0:
            os.replace(MARSHAL + ".tmp", MARSHAL)
            return
    if os.path.exists(MARSHAL):  # of other sources, or another torch
        os.remove(MARSHAL)
    sys.stderr.write(said + "_marshal.so could not be built; the binding's serving calls check "
                            "their arguments in Python instead (6 us a call more)\n")


def build(force: bool = False, verbose: bool = False) -> str:
    lib = force or not _newer_than_inputs(LIB) or not os.path.exists(REPORT)
    beside = _start_marshal() if force or not _marshal_up_to_date() else None
    try:
        if lib:
            cmd = _lib_command()
            res = subprocess.run(cmd, capture_output=True, text=True)
            if res.returncode != 0:
                sys.stderr.write(res.stdout + res.stderr)
                raise subprocess.CalledProcessError(res.returncode, cmd)
            if verbose:
                sys.stderr.write(res.stderr)
            os.makedirs(os.path.dirname(REPORT), exist_ok=True)
            with open(REPORT, "w") as f:
                f.write(res.stderr)
            os.replace(LIB + ".tmp", LIB)
    finally:
        if beside is not None:
            _finish_marshal(*beside)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="--verbose" in sys.argv)
    print(LIB)
