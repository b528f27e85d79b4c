"""Build libproj_gb300 (the C-ABI library) with nvcc for sm_103a, in-tree.

Each translation unit is compiled in parallel; the shared library lands next to
this file as ``libproj_gb300.<machine>.so`` (the machine suffix keeps x86 and
Arm builds apart).  Objects go to ``_build/<machine>/``.  The calls that take
PyTorch tensors (csrc/bind.cpp) are a file of their own beside it, built on first
use; the library and its C ABI need neither PyTorch nor g++.
"""
from __future__ import annotations

import importlib.util
import os
import platform
import shutil
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
SOURCES = ["proj_api.cu", "planner.cpp", "kernel_tc_lean.cu", "kernel_tc_fused.cu", "kernel_tc_pair.cu",
           "kernel_tc_pair_fused.cu", "q4_api.cu", "kv_api.cu"]
HEADERS = [os.path.join(CSRC, "proj_internal.h"), os.path.join(CSRC, "proj_kernel.cuh"),
           os.path.join(CSRC, "proj_aux.cuh"), os.path.join(CSRC, "proj_launch.h"),
           os.path.join(CSRC, "proj_host.h"), os.path.join(CSRC, "proj_warp.cuh"), os.path.join(CSRC, "q4_internal.h"),
           os.path.join(CSRC, "q4_kernels.cuh"), os.path.join(CSRC, "kv_internal.h"),
           os.path.join(CSRC, "kv_append.cuh"), os.path.join(CSRC, "kv_attend.cuh"),
           os.path.join(INCLUDE, "proj.h")]

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
COMMON = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I" + INCLUDE, "-I" + CSRC]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libproj_gb300")


def library_path() -> str:
    return os.path.join(PKG, f"libproj_gb300.{platform.machine()}.so")


def bind_path() -> str:
    """Where _bind lies: one file for each Python and PyTorch, whose binary interfaces it uses."""
    import torch
    return os.path.join(PKG, f"_bind.{sysconfig.get_config_var('SOABI')}.torch-{torch.__version__}.so")


def _torch_dir() -> str:
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        raise RuntimeError("PyTorch not found: its headers are required to build _bind")
    return spec.submodule_search_locations[0]


def _run(cmd, what: str) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _objdir() -> str:
    path = os.path.join(PKG, "_build", platform.machine())
    os.makedirs(path, exist_ok=True)
    return path


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the library (if sources changed) and return its path.  Needs nvcc alone."""
    out = library_path()
    srcs = [os.path.join(CSRC, s) for s in SOURCES]
    if not force and not _stale(out, srcs + HEADERS):
        return out
    objdir = _objdir()

    def compile_one(src):
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        cmd = [nvcc(), *ARCH_FLAGS, *COMMON, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd))
        _run(cmd, f"compiling {src}")
        return obj

    with ThreadPoolExecutor(max_workers=len(srcs)) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = out + f".tmp{os.getpid()}"
    _run([nvcc(), *ARCH_FLAGS, "-shared", "-o", tmp, *objs], "linking libproj_gb300")
    os.replace(tmp, out)
    return out


def build_bind(force: bool = False, verbose: bool = False) -> str:
    """Compile the calls that take PyTorch tensors (if sources changed), next to
    the library that they call, and return their path.  Needs PyTorch and g++."""
    out, src = bind_path(), os.path.join(CSRC, "bind.cpp")
    if not force and not _stale(out, [src, os.path.join(INCLUDE, "proj.h")]):
        build(verbose=verbose)
        return out
    t, gxx = _torch_dir(), shutil.which("g++") or "g++"
    obj = os.path.join(_objdir(), os.path.basename(out) + ".o")
    cmd = [gxx, "-O2", "-std=c++17", "-fPIC", "-I" + INCLUDE, "-I" + sysconfig.get_paths()["include"],
           "-I" + os.path.join(t, "include"), "-I" + os.path.join(t, "include", "torch", "csrc", "api", "include"),
           "-I" + os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"), "-c", src, "-o", obj]
    if verbose:
        print(" ".join(cmd))
    with ThreadPoolExecutor(max_workers=1) as ex:
        compiled = ex.submit(_run, cmd, f"compiling {src}")
        library = build(verbose=verbose)
        compiled.result()
    tmp = out + f".tmp{os.getpid()}"
    _run([gxx, "-shared", "-o", tmp, obj, "-L" + PKG, "-l:" + os.path.basename(library), "-Wl,-rpath,$ORIGIN",
          "-L" + os.path.join(t, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"], "linking _bind")
    os.replace(tmp, out)
    return out


if __name__ == "__main__":
    print(build(force=True, verbose=True))
