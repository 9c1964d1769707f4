"""Builds ``libm3.so`` (the C ABI of include/m3.h) in-tree with nvcc for sm_100a, and
``_m3torch.so``, which hands torch tensors to it, with g++.

Usage: ``python -m state_space_sequence_mamba_b200.build [--force] [-v]``.
No GPU is needed: nvcc cross-compiles.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libm3.so")
TORCH_SRC = os.path.join(CSRC, "m3_torch.cpp")
TORCH_EXT = os.path.join(HERE, "_m3torch.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC",
         "-Xcompiler", "-fvisibility=hidden", "-I", os.path.join(ROOT, "include")]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(
        os.path.join(CSRC, "*.cuh")) + [os.path.join(ROOT, "include", "m3.h"), __file__]
    return any(os.path.getmtime(d) > t for d in deps)


def _ext_stale() -> bool:
    if not os.path.exists(TORCH_EXT):
        return True
    t = os.path.getmtime(TORCH_EXT)
    return any(os.path.getmtime(d) > t for d in (TORCH_SRC, os.path.join(ROOT, "include", "m3.h"), __file__))


def _start_ext(tmp):
    """The g++ process that writes the torch binding to ``tmp``."""
    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(NVCC))
    inc = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), os.path.join(ROOT, "include"), sysconfig.get_paths()["include"]]
    lib = os.path.join(base, "lib")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-I{d}" for d in inc), TORCH_SRC, "-o", tmp, f"-L{lib}",
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    return cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)


def build(force: bool = False, verbose: bool = False) -> str:
    ext = None
    if force or _ext_stale():
        ext_tmp = TORCH_EXT + f".tmp{os.getpid()}"
        ext = _start_ext(ext_tmp)
    try:
        _build_lib(force, verbose)
    finally:
        out, _ = ext[1].communicate() if ext else (b"", None)
    if ext:
        if verbose or ext[1].returncode != 0:
            sys.stdout.write(out.decode())
        if ext[1].returncode != 0:
            raise RuntimeError("g++ failed: " + " ".join(ext[0]))
        os.replace(ext_tmp, TORCH_EXT)
    return LIB


def _build_lib(force: bool, verbose: bool) -> str:
    if not force and not _stale():
        return LIB
    objs = []
    bdir = os.path.join(HERE, "_build")
    os.makedirs(bdir, exist_ok=True)
    procs = []
    for src in sources():
        obj = os.path.join(bdir, os.path.basename(src) + ".o")
        cmd = [NVCC, *ARCH, *FLAGS, "-c", src, "-o", obj]
        if verbose:
            cmd += ["-Xptxas", "-v"]
        procs.append((cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
        objs.append(obj)
    for cmd, pr in procs:
        out, _ = pr.communicate()
        if verbose or pr.returncode != 0:
            sys.stdout.write(out.decode())
        if pr.returncode != 0:
            raise RuntimeError("nvcc failed: " + " ".join(cmd))
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.check_call([NVCC, *ARCH, "-shared", "-o", tmp, *objs])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
