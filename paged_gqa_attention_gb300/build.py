"""Build libpagedattn.so (sm_103a) in-tree with nvcc.

Each .cu file is compiled in parallel with
``-gencode arch=compute_103a,code=sm_103a -O3 -lineinfo`` and the objects are linked
into ``paged_gqa_attention_gb300/libpagedattn.so`` (CUDA runtime linked statically, so
the library loads on a machine without a GPU driver; every compute call then fails
with PA_ERR_CUDA).  Objects go to ``_build/`` at the repository root.  The library needs no PyTorch.

csrc/binding.cpp becomes ``_binding.so`` beside it with g++, once the library stands: it links the
library and PyTorch, and is left out where PyTorch is not installed.  ``_binding.abi`` names the
PyTorch and Python that it was built for; with another one it is built again.
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
BINDING_ABI_PATH = os.path.join(PKG, "_binding.abi")
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


def _torch():
    """PyTorch, or None where it is not installed."""
    try:
        import torch
    except ImportError:
        return None
    return torch


def binding_abi() -> str | None:
    """The PyTorch and Python whose binary interfaces the binding is built against."""
    torch = _torch()
    return torch and f"torch {torch.__version__} {sysconfig.get_config_var('EXT_SUFFIX')}"


def _recorded_abi() -> str | None:
    """What the binding in place was built for, None where that is not known."""
    try:
        with open(BINDING_ABI_PATH) as f:
            return f.read()
    except FileNotFoundError:
        return None


def _older(path: str, inputs) -> bool:
    """Whether path is missing or older than one of the files that it is made of."""
    if not os.path.exists(path):
        return True
    t = os.path.getmtime(path)
    return any(os.path.getmtime(f) > t for f in inputs)


def library_up_to_date() -> bool:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".h"))]
    return not _older(LIB_PATH, files + [os.path.join(INCLUDE, "pagedattn.h"), os.path.abspath(__file__)])


def binding_up_to_date() -> bool:
    if _older(BINDING_PATH, [os.path.join(CSRC, BINDING_SOURCE), os.path.join(INCLUDE, "pagedattn.h"),
                             os.path.abspath(__file__)]):
        return False
    return _recorded_abi() == binding_abi()


def _run(cmd, what: str, verbose: bool = False):
    res = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or res.returncode:
        sys.stderr.write(res.stdout + res.stderr)
    if res.returncode:
        raise RuntimeError(f"{what} failed")


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile and link what is missing or stale of the library and its binding; return the
    library's path."""
    library = force or not library_up_to_date()
    torch = _torch()
    binding = torch is not None and (force or not binding_up_to_date())
    if torch is None:
        sys.stderr.write("PyTorch is not installed: _binding.so is left out\n")
    if not library and not binding:
        return LIB_PATH
    nvcc = _nvcc()
    gxx = shutil.which("g++") or "g++"
    os.makedirs(BUILD_DIR, exist_ok=True)
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.splitext(os.path.basename(src))[0] + ".o")
        if src == BINDING_SOURCE:
            include = os.path.join(os.path.dirname(torch.__file__), "include")
            cmd = [gxx, "-O2", "-std=c++17", "-fPIC", "-I", INCLUDE, "-I", sysconfig.get_paths()["include"],
                   "-I", include, "-I", os.path.join(include, "torch", "csrc", "api", "include"),
                   "-I", os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")]
        else:
            cmd = [nvcc] + NVCC_FLAGS + extra
        _run(cmd + ["-c", os.path.join(CSRC, src), "-o", obj], f"compiling {src}", verbose or ptxas_info)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        bound = ex.submit(compile_one, BINDING_SOURCE) if binding else None
        objects = [ex.submit(compile_one, src) for src in SOURCES] if library else []
    if library:
        tmp = LIB_PATH + f".tmp{os.getpid()}"
        _run([nvcc] + ARCH + ["-shared", "-o", tmp] + [o.result() for o in objects], "linking libpagedattn.so")
        os.replace(tmp, LIB_PATH)
    if binding:
        tmp = BINDING_PATH + f".tmp{os.getpid()}"
        torch_lib = os.path.join(os.path.dirname(torch.__file__), "lib")
        _run([gxx, "-shared", "-o", tmp, bound.result(), "-L", os.path.dirname(LIB_PATH),
              "-l:" + os.path.basename(LIB_PATH), "-L", torch_lib, "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10",
              "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + torch_lib], "linking _binding.so")
        if _recorded_abi() not in (None, binding_abi()):
            os.remove(BINDING_ABI_PATH)      # (it names the old one)
        os.replace(tmp, BINDING_PATH)
        tmp = BINDING_ABI_PATH + f".tmp{os.getpid()}"
        with open(tmp, "w") as f:
            f.write(binding_abi())
        os.replace(tmp, BINDING_ABI_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
