"""Compile the CUDA sources in ``csrc/`` into ``_build/libmoe_nvfp4.so`` (sm_103a only).

Each translation unit is compiled by nvcc in parallel, then linked into one
shared library with the CUDA runtime linked statically.  The driver API entry
point needed for tensor maps is resolved at run time, so the library does not
link libcuda.  ``csrc/binding.cpp``, the Python module with the argument checks
of the operators around the layer, is compiled beside it by g++ against the
installed torch and linked to the library.  The library needs nvcc alone: where
the binding cannot be built (no torch, no Python headers), the library still is,
and build() warns.
Usage: ``python -m nvfp4_quantized_moe_topk_gb300.build``.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libmoe_nvfp4.so")
BINDING = os.path.join(BUILD, "moe_binding.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmoe_nvfp4")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _newer(target: str, inputs: list[str]) -> bool:
    """Whether target is there and no older than its inputs, the header and this file."""
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(p) <= t for p in
               [*inputs, *glob.glob(os.path.join(ROOT, "include", "*.h")), os.path.abspath(__file__)])


def _library_up_to_date() -> bool:
    return _newer(LIB, sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")))


def _binding_up_to_date() -> bool:
    return _newer(BINDING, glob.glob(os.path.join(CSRC, "*.cpp")))


def up_to_date() -> bool:
    return _library_up_to_date() and _binding_up_to_date()


def _torch_dir() -> str:
    import importlib.util

    spec = importlib.util.find_spec("torch")
    if spec is None or spec.origin is None:
        raise RuntimeError("torch is not installed")
    return os.path.dirname(spec.origin)


def _compile_binding() -> str:
    """The object file of csrc/binding.cpp."""
    import sysconfig

    torch, obj = _torch_dir(), os.path.join(BUILD, "binding.cpp.o")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-w", "-I", os.path.join(torch, "include"),
           "-I", os.path.join(torch, "include", "torch", "csrc", "api", "include"), "-I", cuda,
           "-I", sysconfig.get_paths()["include"], "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on binding.cpp:\n{r.stderr}")
    return obj


def _link_binding(obj: str):
    tmp = BINDING + f".tmp{os.getpid()}"
    libs = os.path.join(_torch_dir(), "lib")
    r = subprocess.run(["g++", "-shared", "-o", tmp, obj, "-L", BUILD, "-l:libmoe_nvfp4.so", "-Wl,-rpath,$ORIGIN",
                        "-L", libs, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the binding failed:\n{r.stderr}")
    os.replace(tmp, BINDING)


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    extra = list(extra or [])

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [cc, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stderr}")
        if verbose and r.stderr:
            sys.stderr.write(r.stderr)
        return obj

    library = force or not _library_up_to_date()
    with cf.ThreadPoolExecutor(max_workers=min(16, len(sources()) + 1)) as ex:
        binding = ex.submit(_compile_binding) if force or not _binding_up_to_date() else None
        objs = list(ex.map(compile_one, sources())) if library else []
    if library:
        tmp = LIB + f".tmp{os.getpid()}"
        r = subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stderr}")
        os.replace(tmp, LIB)
    if binding is not None:
        try:
            _link_binding(binding.result())
        except (RuntimeError, OSError) as e:
            if os.path.exists(BINDING):  # of other sources than the library's
                os.remove(BINDING)
            warnings.warn(f"{LIB} is built, the Python calls of the operators around the layer are not: {e}")
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True,
                extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else None))
