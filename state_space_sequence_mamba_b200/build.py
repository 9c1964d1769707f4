"""Builds ``libm3.so`` (the C ABI of include/m3.h) in-tree with nvcc for sm_100a, and
``_m3torch``, which hands torch tensors to it, with g++.

Usage: ``python -m state_space_sequence_mamba_b200.build [--force] [-v] [--lib-only]``.
No GPU is needed: nvcc cross-compiles. ``_m3torch`` needs the headers of Python and torch, and serves the
Python entry points of all but the scan; ``libm3.so`` alone (``--lib-only``, or
what is there when the other fails) serves the C ABI and the scan's Python entry points.
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
TORCH_EXT = os.path.join(HERE, "_m3torch" + sysconfig.get_config_var("EXT_SUFFIX"))
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


def ext_target() -> str:
    """What the torch binding is compiled for, which it also holds as ``built_for``: it is built again, and
    refused, under another torch or Python."""
    import torch
    return f"torch {torch.__version__}, Python {sys.version.split()[0]}"


def _ext_stale() -> bool:
    if not os.path.exists(TORCH_EXT):
        return True
    with open(TORCH_EXT, "rb") as f:
        if ext_target().encode() not in f.read():
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
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DM3_BUILT_FOR="{ext_target()}"',
           *(f"-I{d}" for d in inc), TORCH_SRC, "-o", tmp, f"-L{lib}",
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    return cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)


def build(force: bool = False, verbose: bool = False, ext: bool = True) -> str:
    """Builds what is out of date. Raises if the torch binding (with ``ext``) fails, after the library is there."""
    started = failed = None
    tmp = TORCH_EXT + f".tmp{os.getpid()}"
    try:
        if ext and (force or _ext_stale()):
            started = _start_ext(tmp)
    except (ImportError, OSError) as e:
        failed = e
    try:
        _build_lib(force, verbose)
    finally:
        out, _ = started[1].communicate() if started else (b"", None)
    if started:
        if verbose or started[1].returncode != 0:
            sys.stdout.write(out.decode())
        if started[1].returncode != 0:
            failed = "g++ failed: " + " ".join(started[0])
        else:
            os.replace(tmp, TORCH_EXT)
    if failed:
        raise RuntimeError(f"{LIB} is built, {TORCH_EXT} is not ({failed}): the Python entry points of linear "
                           "attention and the grouped norm need it")
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
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, ext="--lib-only" not in sys.argv))
