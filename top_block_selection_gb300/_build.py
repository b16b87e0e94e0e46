"""Builds libqsa.so in-tree with nvcc for sm_103a (no CMake).

Each translation unit compiles in parallel; the objects link into
``top_block_selection_gb300/lib/libqsa.so`` with the CUDA runtime linked
statically, so the library needs only the NVIDIA driver at run time. Beside it,
``_qsa_kv.so`` is the CPython module through which PyTorch tensors reach the
paged-cache calls (g++, PyTorch's and Python's headers). Where these are not
installed the library is built without it.
Run ``python -m top_block_selection_gb300._build`` or call ``build()``.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIBDIR = os.path.join(HERE, "lib")
OBJDIR = os.path.join(LIBDIR, "obj")
LIBPATH = os.path.join(LIBDIR, "libqsa.so")
BINDINGPATH = os.path.join(LIBDIR, "_qsa_kv.so")
BINDINGSRC = os.path.join(CSRC, "kv_binding.cpp")

SOURCES = ["qsa_runtime.cu", "score_tc.cu", "select.cu", "convert.cu", "fused.cu", "fused_h1.cu",
           "fused_h2.cu", "fused_h4.cu", "fused_h8.cu", "fused_h16.cu", "fused_h32.cu",
           "split_reduce.cu", "split_reduce_static.cu", "kv_append.cu", "kv_attend.cu",
           "kv_attend_many.cu", "kv_attend_d64_t2.cu", "kv_attend_d64_t3.cu", "kv_attend_d128_t2.cu", "kv_attend_d128_t3.cu",
           "qsa_api.cpp"]
HEADERS = ["qsa_device.cuh", "qsa_internal.h", "select_row.cuh", "select_warp.cuh", "fused_kernel.cuh",
           "kv_internal.h", "kv_attend_kernel.cuh", "kv_attend_many.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
COMMON = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libqsa.so")


def _stale(out: str, deps) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def _binding_needs():
    """Why the CPython module cannot be built here, or None."""
    if importlib.util.find_spec("torch") is None:
        return "PyTorch is not installed"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python's headers are not installed"
    return None


def _binding_versions() -> str:
    """What the CPython module was compiled against; it is built anew for others."""
    try:
        torch = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:  # importable, but not installed as a package
        torch = importlib.util.find_spec("torch").origin
    return f"torch {torch}, {sysconfig.get_config_var('EXT_SUFFIX')}\n"


def _binding_stale() -> bool:
    stamp = BINDINGPATH + ".versions"
    if _stale(BINDINGPATH, [BINDINGSRC, __file__, os.path.join(INCLUDE, "qsa.h")]) or not os.path.exists(stamp):
        return True
    with open(stamp) as f:
        return f.read() != _binding_versions()


def _binding_command() -> list:
    """g++ command of the CPython module that marshals PyTorch tensors."""
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    include = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
               os.path.join(cuda, "include"), sysconfig.get_paths()["include"], INCLUDE]
    return ["g++", "-std=c++17", "-O2", "-fPIC", "-shared", *(x for i in include for x in ("-isystem", i)), BINDINGSRC,
            "-o", BINDINGPATH, "-L" + os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def build(verbose: bool = False, extra_flags=()) -> str:
    """Compile (if stale) and return the path of libqsa.so."""
    nvcc = _nvcc()
    os.makedirs(OBJDIR, exist_ok=True)
    hdrs = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(INCLUDE, "qsa.h")]
    jobs = []
    objs = []
    for src in SOURCES:
        sp = os.path.join(CSRC, src)
        op = os.path.join(OBJDIR, src + ".o")
        objs.append(op)
        if _stale(op, [sp, __file__] + hdrs):
            jobs.append([nvcc, *ARCH, *COMMON, *extra_flags, "-c", sp, "-o", op])
    missing = _binding_needs()
    binding = missing is None and _binding_stale()
    if missing:
        sys.stderr.write(f"{os.path.basename(BINDINGPATH)} not built: {missing}\n")
    if binding:
        jobs.append(_binding_command())
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=len(jobs)) as ex:
            for cmd, res in zip(jobs, ex.map(lambda c: subprocess.run(c, capture_output=True, text=True), jobs)):
                if verbose and (res.stdout or res.stderr):
                    sys.stderr.write(res.stdout + res.stderr)
                if res.returncode != 0:
                    raise RuntimeError("compilation failed:\n" + " ".join(cmd) + "\n" + res.stdout + res.stderr)
    if binding:
        with open(BINDINGPATH + ".versions", "w") as f:
            f.write(_binding_versions())
    if jobs or _stale(LIBPATH, objs):
        cmd = [nvcc, *ARCH, "-shared", "-o", LIBPATH, *objs, "-lrt", "-ldl", "-lpthread"]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError("link failed:\n" + " ".join(cmd) + "\n" + res.stdout + res.stderr)
    return LIBPATH


if __name__ == "__main__":
    print(build(verbose=True))
