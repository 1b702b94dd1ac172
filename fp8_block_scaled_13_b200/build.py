"""Build the CUDA library libpuro_fp8.so (nvcc, sm_100a only) and the compiled
wrappers _binding.so (g++, against torch) in-tree."""
from __future__ import annotations

import importlib.metadata
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB_PATH = os.path.join(HERE, "libpuro_fp8.so")
SOURCES = ["puro_fp8.cu"]
DEPS = ["puro_fp8.cu", "common.cuh", "quant.cuh", "gemm.cuh", "norm.cuh", "gated.cuh",
        "ortho.cuh", "ortho_small.cuh"]
HEADER = os.path.join(ROOT, "include", "puro_fp8.h")
BINDING_PATH = os.path.join(HERE, "_binding.so")
BINDING_SOURCE = os.path.join(CSRC, "binding.cpp")
BINDING_TARGET_PATH = os.path.join(HERE, "_binding.target")  # the interpreter and torch that _binding.so is for


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA library cannot be built")


def nvcc_command(out: str, verbose_ptxas: bool = False) -> list:
    cmd = [
        nvcc_path(),
        "-gencode", "arch=compute_100a,code=sm_100a",
        "-O3", "-lineinfo", "-std=c++17",
        "-Xcompiler", "-fPIC,-fvisibility=hidden",
        "-shared", "-Xlinker", "--exclude-libs,ALL",
        "-o", out,
    ]
    if verbose_ptxas:
        cmd += ["-Xptxas", "-v"]
    cmd += [os.path.join(CSRC, s) for s in SOURCES]
    return cmd


def binding_command(out: str) -> list:
    import torch

    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc_path())))
    base = os.path.dirname(torch.__file__)
    include = [os.path.join(base, "include"), os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
            "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI, "-o", out, BINDING_SOURCE,
            *("-I" + d for d in include), "-L" + HERE, "-l:" + os.path.basename(LIB_PATH),
            "-L" + os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]


def _stale(out: str, deps: list) -> bool:
    return not os.path.exists(out) or any(os.path.getmtime(d) > os.path.getmtime(out) for d in deps)


def stale() -> bool:
    return _stale(LIB_PATH, [os.path.join(CSRC, d) for d in DEPS] + [HEADER])


def binding_target() -> str:
    return "%s torch %s\n" % (sysconfig.get_config_var("SOABI"), importlib.metadata.version("torch"))


def binding_stale() -> bool:
    if _stale(BINDING_PATH, [BINDING_SOURCE, HEADER]):
        return True
    try:
        with open(BINDING_TARGET_PATH) as f:
            return f.read() != binding_target()
    except OSError:
        return True


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    if force or stale():
        tmp = LIB_PATH + ".tmp%d" % os.getpid()
        subprocess.run(nvcc_command(tmp, verbose_ptxas), check=True)
        os.replace(tmp, LIB_PATH)
    if force or binding_stale():
        tmp = BINDING_PATH + ".tmp%d" % os.getpid()
        subprocess.run(binding_command(tmp), check=True)
        os.replace(tmp, BINDING_PATH)
        tmp = BINDING_TARGET_PATH + ".tmp%d" % os.getpid()
        with open(tmp, "w") as f:
            f.write(binding_target())
        os.replace(tmp, BINDING_TARGET_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose_ptxas=True))
