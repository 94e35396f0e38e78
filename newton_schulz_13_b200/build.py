"""Builds, in-tree, libmuon.so (the sm_100a kernels and the C ABI) with nvcc, and _plain.*.so (the plain
case of the gradient operators' Python calls, csrc/binding.cpp) with g++."""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libmuon.so")
SOURCES = ["api.cu", "elementwise.cu", "ns_gemm.cu", "ns_gemm_x3.cu", "noalloc.cu",
           "ops_api.cu", "embedding.cu", "rmsnorm.cu", "checkpoint.cu", "weight_grad.cu"]
HEADERS = ["muon_internal.h", "ptx.cuh", "tile_sched.cuh", "device_once.h", "pair_pipe.cuh",
           "ops_internal.h", "vec_io.cuh", "mx.cuh", "fast_div.cuh"]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-shared",
]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def sources():
    return [os.path.join(CSRC, s) for s in SOURCES]


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(ROOT, "include", "muon.h")]
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    if not force and not stale():
        return LIB
    cmd = [_nvcc(), *NVCC_FLAGS, *extra, "-I", os.path.join(ROOT, "include"), *sources(), "-o", LIB]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.check_call(cmd)
    return LIB


def binding_path() -> str:
    """Where the extension lies that was built for this interpreter and this torch, whose layouts it
    holds: one that was built for others has another name."""
    import sysconfig

    import torch
    version = f"{torch.__version__}-{str(torch.version.git_version)[:8]}-{int(torch._C._GLIBCXX_USE_CXX11_ABI)}"
    return os.path.join(HERE, f"_plain.{sysconfig.get_config_var('SOABI')}.torch-{version}.so")


def binding_stale() -> bool:
    path = binding_path()
    if not os.path.exists(path):
        return True
    t = os.path.getmtime(path)
    return any(os.path.getmtime(d) > t for d in (os.path.join(CSRC, "binding.cpp"), os.path.join(ROOT, "include", "muon.h")))


def build_binding(force: bool = False, verbose: bool = False) -> str:
    path = binding_path()
    if not force and not binding_stale():
        return path
    import sysconfig

    import torch
    home = os.path.dirname(torch.__file__)
    inc, libs = os.path.join(home, "include"), os.path.join(home, "lib")
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    out = f"{path}.{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", "-Wno-attributes",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", cuda,
           "-isystem", sysconfig.get_paths()["include"], os.path.join(CSRC, "binding.cpp"), "-o", out,
           "-L", libs, "-lc10", "-lc10_cuda", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", f"-Wl,-rpath,{libs}"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.check_call(cmd)
    os.replace(out, path)
    return path


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra=["-Xptxas", "-v"] if "--ptxas" in sys.argv else [])
    build_binding(force="--force" in sys.argv, verbose=True)
