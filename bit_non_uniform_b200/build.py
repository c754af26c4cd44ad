"""Build libcq.so (the CUDA library) in-tree with nvcc for sm_100a, and
_cq_torch.so (its INT8 calls on torch tensors, host code) with g++.

    python -m bit_non_uniform_b200.build
"""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libcq.so")
SOURCES = ["cq_lib.cu"]
HEADERS = ["cq_gemv.cuh", "cq_gemv_launch.cuh", "cq_narrow.cuh", "cq_narrow_launch.cuh", "cq_api.cu", "cq_gemm.cu", "cq_moe.cu", "cq_noalloc.cu", "cq_a8.cu", "cq_a8.cuh", "cq_device.cuh", "cq_engine.cuh",
           "cq_i8.cu", "cq_i8.cuh", "cq_i8_tc.cuh", "cq_i8_group.cuh", "cq_route.cu", "cq_route.cuh",
           "cq_host.h"]
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-rdc=false",
]


TORCH_SRC = os.path.join(CSRC, "cq_torch.cpp")
TORCH_LIB = os.path.join(HERE, "_cq_torch.so")
CXX = os.environ.get("CXX", "g++")


def built_for() -> str:
    """The torch and Python whose C++ and C interfaces the extension uses.  The
    extension carries this line, and one that carries another is not loaded."""
    import torch
    return f"torch {torch.__version__}, python {sys.version_info[0]}.{sys.version_info[1]}"


def _torch_stale() -> bool:
    if not os.path.exists(TORCH_LIB):
        return True
    t = os.path.getmtime(TORCH_LIB)
    if any(os.path.getmtime(d) > t for d in (TORCH_SRC, os.path.join(INCLUDE, "cq.h"))):
        return True
    with open(TORCH_LIB, "rb") as f:
        return built_for().encode() not in f.read()


def build_torch(force: bool = False) -> str | None:
    """The extension links against libcq.so beside it.  libcq and the binding
    are complete without it (its calls then go through Python), so that a
    compiler that fails here is reported and fails nothing else; the extension
    of older sources is taken away."""
    if not force and not _torch_stale():
        return TORCH_LIB
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(NVCC))
    tmp = TORCH_LIB + f".tmp{os.getpid()}"
    try:
        subprocess.check_call([
            CXX, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            f'-DCQ_BUILT_FOR="{built_for()}"',
            "-I", INCLUDE, "-I", sysconfig.get_paths()["include"],
            "-I", os.path.join(root, "include"),
            "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"),
            "-I", os.path.join(cuda, "include"), TORCH_SRC, "-o", tmp,
            "-L", HERE, "-l:libcq.so", "-Wl,-rpath,$ORIGIN", "-L", os.path.join(root, "lib"),
            "-ltorch_python", "-ltorch", "-ltorch_cuda", "-ltorch_cpu", "-lc10", "-lc10_cuda"])
    except (OSError, subprocess.CalledProcessError) as e:
        print(f"{os.path.basename(TORCH_LIB)} was not built: {e}", file=sys.stderr)
        for path in (tmp, TORCH_LIB):
            if os.path.exists(path):
                os.remove(path)
        return None
    os.replace(tmp, TORCH_LIB)
    return TORCH_LIB


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + [
        os.path.join(INCLUDE, h) for h in ("cq.h", "cq_hooks.h", "cq_hooks_i8.h")]
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        build_torch()
        return LIB
    objs = []
    build_dir = os.path.join(HERE, "_build")
    os.makedirs(build_dir, exist_ok=True)
    for src in SOURCES:
        obj = os.path.join(build_dir, src.replace(".cu", ".o"))
        cmd = [NVCC, *FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd += ["-Xptxas", "-v"]
        subprocess.check_call(cmd)
        objs.append(obj)
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.check_call([NVCC, "-shared", "-gencode", "arch=compute_100a,code=sm_100a",
                           *objs, "-o", tmp, "-lcuda"])
    os.replace(tmp, LIB)
    build_torch(force)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
