"""Build libnvfp4.so in-tree with nvcc for sm_100a (cross-compiles without a GPU), and the
torch binding beside it with the host compiler.

    python -m nvfp4_w4a4_quantized_08_b200.build [--verbose]
"""
from __future__ import annotations

import glob
import os
import re
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libnvfp4.so")
BINDING = os.path.join(HERE, "_binding.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    # IEEE binary32: no flush-to-zero, correctly rounded division / sqrt
    "-ftz=false", "-prec-div=true", "-prec-sqrt=true",
]


# Kernels whose warps share out their registers anew, which adds up only with this many a thread at
# launch: a compiler that gives another number must not go unnoticed until the first call fails.
LAUNCH_REGISTERS = {"chunk_kernel": 128}


def check_registers(ptxas_log: str) -> None:
    """Raises if a kernel of LAUNCH_REGISTERS is missing from the output of ptxas -v, or
    uses another number of registers."""
    found = re.findall(r"entry function '(\S+)'.*?Used (\d+) registers", ptxas_log, re.DOTALL)
    for name, want in LAUNCH_REGISTERS.items():
        used = {int(n) for symbol, n in found if name in symbol}
        if used != {want}:
            raise RuntimeError(f"{name} has to be compiled to {want} registers a thread, not "
                               f"{sorted(used)}: its register split does not add up")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def deps():
    return sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh")) +
                              glob.glob(os.path.join(CSRC, "*.h")) +
                              [os.path.join(os.path.dirname(HERE), "include", "nvfp4.h")])


def _newer(out: str, inputs) -> bool:
    if not os.path.exists(out):
        return False
    t = os.path.getmtime(out)
    return all(os.path.getmtime(f) <= t for f in inputs)


def up_to_date() -> bool:
    return _newer(LIB, deps())


def build_binding(force: bool = False) -> str:
    import sysconfig

    import torch

    src = os.path.join(CSRC, "binding.cpp")
    header = os.path.join(os.path.dirname(HERE), "include", "nvfp4.h")
    # the C++ interfaces of torch and Python it is compiled against, noted beside it
    built_for = f"torch {torch.__version__}, {sysconfig.get_config_var('SOABI')}\n"
    stamp = BINDING + ".torch"
    if not force and _newer(BINDING, [src, header]) and os.path.exists(stamp):
        with open(stamp) as f:
            if f.read() == built_for:
                return BINDING
    from torch.utils import cpp_extension

    lib_dir = os.path.join(os.path.dirname(torch.__file__), "lib")
    includes = cpp_extension.include_paths() + [
        sysconfig.get_paths()["include"],
        os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include")]
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           f'-DNVFP4_TORCH_VERSION="{torch.__version__}"',
           *[f"-isystem{i}" for i in includes], src, "-o", tmp, f"-L{lib_dir}",
           f"-Wl,-rpath,{lib_dir}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10",
           "-lc10_cuda", "-ldl"]
    subprocess.run(cmd, check=True)
    os.replace(tmp, BINDING)
    with open(stamp, "w") as f:
        f.write(built_for)
    return BINDING


def build_library(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [NVCC, "-Xptxas=-v", *FLAGS, "-shared", "-o", tmp, *sources()]
    run = subprocess.run(cmd, stderr=subprocess.PIPE, text=True)
    if verbose or run.returncode != 0 or "warning" in run.stderr:
        sys.stderr.write(run.stderr)
    run.check_returncode()
    try:
        check_registers(run.stderr)
    except RuntimeError:
        os.remove(tmp)
        raise
    os.replace(tmp, LIB)
    return LIB


def build(force: bool = False, verbose: bool = False) -> str:
    build_library(force, verbose)   # first: it needs no Python or torch headers
    build_binding(force)
    return LIB


if __name__ == "__main__":
    build(force=True, verbose="--verbose" in sys.argv)
    print(LIB)
