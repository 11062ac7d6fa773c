"""Build libmxq.so in-tree with nvcc for sm_100a, and the torch module _ops.so beside it with g++.

    python -m block_scaled_microscaling_b200.build [--force] [--verbose]

Compiles every .cu file of csrc/ into one shared library next to this file,
with the CUDA runtime linked statically (no dependence on the runtime that
PyTorch ships). -Xptxas -v output (registers, spills, shared memory) goes to
build_ptxas.txt beside the library when --verbose is given.
"""
import glob
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmxq.so")
OPS_SRC = os.path.join(CSRC, "ops_torch.cpp")
OPS = os.path.join(HERE, "_ops.so")

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3", "-std=c++17",
         "-shared", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "-cudart", "static", "--threads", "0", "-I", os.path.join(ROOT, "include")]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _older(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _stale():
    return _older(LIB, sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) +
                  glob.glob(os.path.join(ROOT, "include", "*.h")))


def build_ops(force=False):
    """_ops.so (ops_torch.cpp against the installed torch and libmxq.so)."""
    if not force and not _older(OPS, [OPS_SRC, __file__] + glob.glob(os.path.join(ROOT, "include", "*.h"))):
        return OPS
    import sysconfig

    import torch
    from torch.utils import cpp_extension as ext

    inc = [*ext.include_paths(), os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include"),
           sysconfig.get_path("include")]
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-DTORCH_API_INCLUDE_EXTENSION_H",
           *(a for i in inc for a in ("-isystem", i)), OPS_SRC, "-o", OPS + ".tmp", "-L", HERE, "-l:libmxq.so",
           "-Wl,-rpath,$ORIGIN", "-L", libs, "-ltorch", "-ltorch_cpu", "-ltorch_python", "-lc10", "-lc10_cuda",
           # torch's own C++ library and no other: a compiler that has only the static one would put a second copy into
           # the process, where the first exception with a number in its message ends it
           "-nostdlib++", "-l:libstdc++.so.6"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("g++ failed building _ops.so")
    os.replace(OPS + ".tmp", OPS)
    return OPS


def build(force=False, verbose=False):
    if not force and not _stale():
        build_ops()
        return LIB
    cmd = [NVCC, *FLAGS, *sources(), "-o", LIB + ".tmp"]
    if verbose:
        cmd[1:1] = ["-Xptxas", "-v"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("nvcc failed building libmxq.so")
    if verbose:
        with open(os.path.join(HERE, "build_ptxas.txt"), "w") as f:
            f.write(res.stdout + res.stderr)
    os.replace(LIB + ".tmp", LIB)
    build_ops(force)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
