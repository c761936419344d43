"""Build libpagedattn.so (sm_103a) in-tree with nvcc.

csrc/binding.cpp becomes ``_binding.so`` beside it with g++ (PyTorch's headers; it links the library).
Each .cu file is compiled in parallel with
``-gencode arch=compute_103a,code=sm_103a -O3 -lineinfo`` and the objects are linked
into ``paged_gqa_attention_gb300/libpagedattn.so`` (CUDA runtime linked statically, so
the library loads on a machine without a GPU driver; every compute call then fails
with PA_ERR_CUDA).  Objects go to ``_build/`` at the repository root.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_PATH = os.path.join(PKG, "libpagedattn.so")
BINDING_PATH = os.path.join(PKG, "_binding.so")
BINDING_SOURCE = "binding.cpp"
SOURCES = ["api.cu", "kv_append.cu", "decode.cu", "decode_fp8.cu", "prefill.cu", "qkv.cu",
           "rope_append.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpagedattn.so")


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".h", ".cpp"))]
    files.append(os.path.join(INCLUDE, "pagedattn.h"))
    files.append(os.path.abspath(__file__))
    return files


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH) or not os.path.exists(BINDING_PATH):
        return False
    t = min(os.path.getmtime(LIB_PATH), os.path.getmtime(BINDING_PATH))
    return all(os.path.getmtime(f) <= t for f in _inputs())


def _torch_dir() -> str:
    import torch

    return os.path.dirname(torch.__file__)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile and link the library if it is missing or stale; return its path."""
    if not force and up_to_date():
        return LIB_PATH
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    gxx = shutil.which("g++") or "g++"
    torch_dir = _torch_dir()
    torch_include = os.path.join(torch_dir, "include")

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
        if src == BINDING_SOURCE:
            cmd = [gxx, "-O2", "-std=c++17", "-fPIC", "-I", INCLUDE, "-I", sysconfig.get_paths()["include"],
                   "-I", torch_include, "-I", os.path.join(torch_include, "torch", "csrc", "api", "include"),
                   "-I", os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")]
        else:
            cmd = [nvcc] + NVCC_FLAGS + extra
        cmd += ["-c", os.path.join(CSRC, src), "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, res

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        results = list(ex.map(compile_one, SOURCES + [BINDING_SOURCE]))
    for src, _, res in results:
        if verbose or ptxas_info or res.returncode:
            sys.stderr.write(res.stdout + res.stderr)
        if res.returncode:
            raise RuntimeError(f"compiling {src} failed")
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc] + ARCH + ["-shared", "-o", tmp] + [obj for src, obj, _ in results if src != BINDING_SOURCE]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("linking libpagedattn.so failed")
    os.replace(tmp, LIB_PATH)
    tmp = BINDING_PATH + f".tmp{os.getpid()}"
    torch_lib = os.path.join(torch_dir, "lib")
    cmd = [gxx, "-shared", "-o", tmp, results[-1][1], "-L", PKG, "-l:" + os.path.basename(LIB_PATH), "-L", torch_lib,
           "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + torch_lib]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("linking _binding.so failed")
    os.replace(tmp, BINDING_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
