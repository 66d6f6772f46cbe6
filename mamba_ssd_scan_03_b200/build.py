"""Build libssd.so (the sm_100a CUDA library behind include/ssd.h) and the Python binding of its
served forms (_binding.<Python>.<torch>.so) in-tree.

``python -m mamba_ssd_scan_03_b200.build`` or ``build()``.  One nvcc invocation on the single
translation unit ``csrc/ssd_lib.cu`` and one of the host compiler on ``csrc/binding.cpp``; both land
next to this file so that they travel with the repository snapshot and are loaded from here.
"""
import os
import subprocess
import sys

from . import BINDING_PATH as BINDING

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libssd.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
CXX = os.environ.get("CXX", "g++")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def sources():
    out = [os.path.join(ROOT, "include", "ssd.h")]
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".cu", ".cuh")):
            out.append(os.path.join(CSRC, name))
    return out


def up_to_date(path, deps):
    if not os.path.exists(path):
        return False
    t = os.path.getmtime(path)
    return all(os.path.getmtime(d) <= t for d in deps)


def build_binding(force=False, verbose=False):
    src = os.path.join(CSRC, "binding.cpp")
    if not force and up_to_date(BINDING, [src, os.path.join(ROOT, "include", "ssd.h")]):
        return BINDING
    import sysconfig

    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(NVCC))
    include = [os.path.join(base, "include"),
               os.path.join(base, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = [CXX, "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", "-w",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[f"-I{p}" for p in include], src, "-L" + os.path.join(base, "lib"), "-ltorch_python",
           "-ltorch_cpu", "-lc10", "-lc10_cuda", "-ldl", "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, BINDING)
    return BINDING


def build(force=False, verbose=False, ptxas_info=False):
    build_binding(force, verbose)
    deps = sources()
    if not force and up_to_date(LIB, deps):
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [NVCC, *ARCH, "-O3", "-lineinfo", "-std=c++17", "-shared", "-Xcompiler", "-fPIC",
           "-I", os.path.join(ROOT, "include"), os.path.join(CSRC, "ssd_lib.cu"), "-o", tmp]
    if ptxas_info:
        cmd.insert(1, "-Xptxas=-v")
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="-v" in sys.argv))
