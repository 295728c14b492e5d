"""Builds libexact_topk.so in-tree for sm_103a (nvcc + g++, no CMake).

The CUDA translation units and the host sources compile in parallel; the shared
library links the CUDA runtime dynamically so that it shares one runtime (and
its streams) with PyTorch in the same process.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIBRARY = os.path.join(BUILD_DIR, "libexact_topk.so")

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
CUDA_SOURCES = ["topk_kernels.cu", "cache_kernels.cu", "score_kernels.cu",
                "attention_kernels.cu", "prompt_attention_kernels.cu", "prompt_pair_kernels.cu",
                "cache4_kernels.cu",
                "rotary_kernels.cu", "table_kernels.cu"]
HOST_SOURCES = ["exact_topk_api.cpp", "cache_api.cpp", "batch_api.cpp"]
HEADERS = ["etk_internal.h", "cache_internal.h", "batch_internal.h", "cache_device.cuh",
           "tensor_device.cuh", "prompt_device.cuh"]
PUBLIC_HEADERS = ["exact_topk.h", "exact_topk_cache.h"]


def cuda_home() -> str:
    home = os.environ.get("CUDA_HOME") or os.environ.get("CUDA_PATH")
    if home and os.path.isdir(home):
        return home
    nvcc = shutil.which("nvcc")
    if nvcc:
        return os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    return "/usr/local/cuda"


def _inputs():
    files = [os.path.join(CSRC, s) for s in CUDA_SOURCES + HOST_SOURCES + HEADERS]
    files += [os.path.join(INCLUDE, h) for h in PUBLIC_HEADERS]
    files.append(os.path.abspath(__file__))
    return files


def _stale() -> bool:
    if not os.path.exists(LIBRARY):
        return True
    t = os.path.getmtime(LIBRARY)
    return any(os.path.getmtime(f) > t for f in _inputs())


def _run(cmd):
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("build step failed: " + " ".join(cmd))
    return res.stdout + res.stderr


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compiles the library if any input changed; returns its path."""
    if not force and not _stale():
        return LIBRARY
    os.makedirs(BUILD_DIR, exist_ok=True)
    home = cuda_home()
    nvcc = os.path.join(home, "bin", "nvcc")
    if not os.path.exists(nvcc):
        nvcc = "nvcc"
    inc = ["-I", INCLUDE, "-I", CSRC]
    cu_cmd = [nvcc, *ARCH_FLAGS, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
              "--expt-relaxed-constexpr", *inc]
    if verbose_ptxas:
        cu_cmd.insert(1, "-Xptxas=-v")
    host_cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", *inc,
                "-I", os.path.join(home, "include")]
    cmds, objects = [], []
    for cmd, sources in ((cu_cmd, CUDA_SOURCES), (host_cmd, HOST_SOURCES)):
        for source in sources:
            obj = os.path.join(BUILD_DIR, os.path.splitext(source)[0] + ".o")
            cmds.append([*cmd, "-c", os.path.join(CSRC, source), "-o", obj])
            objects.append(obj)
    with ThreadPoolExecutor(len(cmds)) as ex:
        outs = list(ex.map(_run, cmds))
    tmp = LIBRARY + f".tmp{os.getpid()}"
    libdir = os.path.join(home, "lib64")
    _run([nvcc, *ARCH_FLAGS, "-shared", "-cudart", "shared", *objects, "-o", tmp,
          "-Xlinker", f"-rpath={libdir}"])
    os.replace(tmp, LIBRARY)
    if verbose_ptxas:
        sys.stdout.write("".join(outs))
    return LIBRARY


if __name__ == "__main__":
    print(build(force=True, verbose_ptxas="-v" in sys.argv))
