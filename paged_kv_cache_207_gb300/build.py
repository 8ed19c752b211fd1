"""Build the CUDA library ``libpaged_kv.so`` in-tree with nvcc for sm_103a.

Translation units compile in parallel into ``_build/`` at the repository root
and link into ``paged_kv_cache_207_gb300/libpaged_kv.so`` (the CUDA runtime is
linked statically).  Run ``python -m paged_kv_cache_207_gb300.build``.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import importlib.util
import os
import re
import shlex
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libpaged_kv.so")
# the quick way through the Python bindings (csrc/pa_binding.cpp), for this interpreter
QUICK = os.path.join(PKG, "_quick.so")
PYTHON_INCLUDE = sysconfig.get_paths()["include"]
_torch = importlib.util.find_spec("torch")
TORCH = _torch.submodule_search_locations[0] if _torch and _torch.submodule_search_locations else None

SOURCES = ["pa_api.cu", "pa_decode.cu", "pa_append.cu", "pa_prefill.cu", "pa_noalloc.cu",
           "pa_rope.cu", "pa_window_decode.cu", "pa_block_manager.cpp"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpaged_kv.so")
    return cand


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "pa.h"))
    files.append(os.path.abspath(__file__))
    if TORCH is not None:
        files.append(os.path.join(TORCH, "version.py"))      # (_quick.so is compiled for one torch)
    return files


def _has_headers() -> bool:
    """Those that csrc/pa_binding.cpp is compiled with: Python's and torch's."""
    return TORCH is not None and all(os.path.exists(f) for f in (
        os.path.join(PYTHON_INCLUDE, "Python.h"), os.path.join(TORCH, "include", "torch", "csrc", "autograd", "python_variable.h"),
        os.path.join(TORCH, "lib", "libc10_cuda.so")))


def _torch_version() -> str:
    with open(os.path.join(TORCH, "version.py")) as f:
        return re.search(r"__version__ = ['\"](.+?)['\"]", f.read()).group(1)


def _stale(made: str) -> bool:
    if not os.path.exists(made):
        return True
    t = os.path.getmtime(made)
    return any(os.path.getmtime(f) > t for f in _inputs())


def _compile(src: str, ptxas_verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [_nvcc(), "-c", src, "-o", obj, "-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
           "-I", INCLUDE, "-I", CSRC] + ARCH
    # optional extra flags, e.g. -DPA_DECODE_WARPS=8 -DPA_DECODE_STAGES=2 for tuning builds
    cmd += os.environ.get("PA_EXTRA_NVCC_FLAGS", "").split()
    if src.endswith(".cu"):
        cmd += ["--expt-relaxed-constexpr"]
        if ptxas_verbose:
            cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    if ptxas_verbose and r.stderr:
        sys.stderr.write(r.stderr)
    return obj


def _compile_quick() -> str | None:
    """csrc/pa_binding.cpp with the C++ compiler (``CXX`` may be a command with arguments), as a
    file to be renamed to QUICK.  None where that does not work, which is said on stderr: the
    bindings do without."""
    tmp = os.path.join(BUILD, f"_quick{os.getpid()}.so")
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    cmd = shlex.split(os.environ.get("CXX", "")) or ["g++"]
    cmd += ["-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            f'-DPA_TORCH_VERSION="{_torch_version()}"', "-I", INCLUDE,
            "-I", PYTHON_INCLUDE, "-isystem", os.path.join(TORCH, "include"),
            "-isystem", os.path.join(TORCH, "include", "torch", "csrc", "api", "include"), "-isystem", cuda,
            os.path.join(CSRC, "pa_binding.cpp"), "-L", os.path.join(TORCH, "lib"), "-ltorch_python", "-ltorch_cpu",
            "-lc10", "-lc10_cuda", "-o", tmp]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
        why = f"{r.stdout}\n{r.stderr}" if r.returncode != 0 else ""
    except OSError as e:
        why = str(e)
    if why:
        sys.stderr.write(f"{cmd[0]} failed on pa_binding.cpp, calls go through Python:\n{why}\n")
        return None
    return tmp


def build(force: bool = False, ptxas_verbose: bool = False) -> str:
    lib = force or ptxas_verbose or _stale(LIB)
    short_cut = _has_headers() and (force or ptxas_verbose or _stale(QUICK))
    if not lib and not short_cut:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    srcs = [os.path.join(CSRC, s) for s in SOURCES] if lib else []
    with cf.ThreadPoolExecutor(max_workers=len(srcs) + 1) as ex:
        quick = ex.submit(_compile_quick) if short_cut else None
        objs = list(ex.map(lambda s: _compile(s, ptxas_verbose), srcs))
    if lib:
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [_nvcc(), "-shared", "-o", tmp] + objs + ARCH + ["-Xcompiler", "-fPIC"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    if quick is not None:
        made = quick.result()
        if made is not None:
            os.replace(made, QUICK)
        elif os.path.exists(QUICK):
            os.remove(QUICK)                     # (of other sources: it must not meet this library)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--ptxas-verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, ptxas_verbose=a.ptxas_verbose))
