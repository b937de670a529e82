"""Builds libdwconv.so in-tree with nvcc for sm_103a.

Each translation unit under ``csrc/`` compiles in parallel to an object file,
then nvcc links them into ``depthwise_convolution_gb300/libdwconv.so`` (CUDA
runtime linked statically).  ``-Xptxas -v`` output is kept in
``_build/ptxas.log`` (registers, spills, shared memory per kernel).
``csrc/torch_ops.cpp`` (the token mixer's calls on PyTorch tensors, with their
autograd nodes) compiles beside them with g++ and becomes ``libdwconv_torch.so``,
a Python extension module linked to the first; without PyTorch the C library is
built alone.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libdwconv.so")
OPS_SRC = os.path.join(CSRC, "torch_ops.cpp")
OPS = os.path.join(PKG, "libdwconv_torch.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
                     "-Xptxas", "-v", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libdwconv")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + [os.path.join(INCLUDE, "dwconv.h"), OPS_SRC,
                                                                   os.path.abspath(__file__)]


def _torch():
    try:
        import torch
    except ImportError:
        return None
    return torch


def needs_build() -> bool:
    made = [LIB] if _torch() is None else [LIB, OPS]
    if not all(os.path.exists(p) for p in made):
        return True
    t = min(os.path.getmtime(p) for p in made)
    return any(os.path.getmtime(p) > t for p in _deps())


def _compile_ops() -> tuple | None:
    import sysconfig

    torch = _torch()
    if torch is None:
        return None
    at = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    obj = os.path.join(BUILD, "torch_ops.o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", INCLUDE]
    for path in (f"{at}/include", f"{at}/include/torch/csrc/api/include", cuda,
                 sysconfig.get_paths()["include"]):
        cmd += ["-isystem", path]
    r = subprocess.run(cmd + ["-c", OPS_SRC, "-o", obj], capture_output=True, text=True)
    link = ["-L", os.path.join(at, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python"]
    return OPS_SRC, [obj] + link, r.returncode, r.stdout + r.stderr


def _compile(src: str) -> tuple:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc()] + NVCC_FLAGS + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    return src, obj, r.returncode, r.stdout + r.stderr


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link libdwconv.so if any source is newer; returns its path."""
    if not force and not needs_build():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(os.cpu_count() or 8, len(srcs) + 1)) as ex:
        ops = ex.submit(_compile_ops)
        results = list(ex.map(_compile, srcs))
    log, made = [], ops.result()
    for src, obj, rc, out in results:
        log.append(f"==== {os.path.basename(src)}\n{out}")
        if rc != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{out}")
    if made is not None and made[2] != 0:
        raise RuntimeError(f"g++ failed on {os.path.basename(made[0])}:\n{made[3]}")
    with open(os.path.join(BUILD, "ptxas.log"), "w") as f:
        f.write("\n".join(log))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc()] + ARCH + ["-shared", "-o", tmp] + [o for _, o, _, _ in results]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}{r.stderr}")
    os.replace(tmp, LIB)
    if made is not None:
        obj, *libs = made[1]
        tmp = OPS + f".tmp{os.getpid()}"
        r = subprocess.run(["g++", "-shared", "-o", tmp, obj, "-L", PKG, "-ldwconv", *libs, "-Wl,-rpath,$ORIGIN"],
                           capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ link failed:\n{r.stdout}{r.stderr}")
        os.replace(tmp, OPS)
    if verbose:
        print("\n".join(log))
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
