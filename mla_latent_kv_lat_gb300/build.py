"""Build libmla.so in-tree from csrc/*.cu with nvcc for sm_103a (GB300), and beside it the module that
takes the paged calls from Python to it (csrc/calls.cpp, against the installed PyTorch; without g++ or a PyTorch with
CUDA it is left out, and the binding makes these calls by itself).

Usage: ``python -m mla_latent_kv_lat_gb300.build [--force]``.  Translation
units compile in parallel; the library links against the shared CUDA runtime
so that it shares one runtime with PyTorch in the same process.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmla.so")
INCLUDE = os.path.join(os.path.dirname(PKG), "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE,
                 "--expt-relaxed-constexpr", "-Xptxas", "-warn-spills"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmla")


def calls_path() -> str:
    """The module of csrc/calls.cpp for this Python and PyTorch."""
    import torch
    version = "".join(c if c.isalnum() else "_" for c in torch.__version__)
    return os.path.join(PKG, f"_calls_{version}{sysconfig.get_config_var('EXT_SUFFIX')}")


def _torch_root() -> str:
    return os.path.dirname(importlib.util.find_spec("torch").origin)


def can_build_calls() -> bool:
    return shutil.which("g++") is not None and os.path.exists(os.path.join(_torch_root(), "lib", "libc10_cuda.so"))


def _build_calls() -> str:
    root = _torch_root()
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    out = calls_path()
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include"), INCLUDE]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", os.path.join(CSRC, "calls.cpp"), "-o", out + ".tmp"]
    for i in inc:
        cmd += ["-isystem" if i != INCLUDE else "-I", i]
    cmd += ["-L" + os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-ldl"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for calls.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(out + ".tmp", out)
    return out


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(CSRC, "*.cpp")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def up_to_date() -> bool:
    made = [LIB] + ([calls_path()] if can_build_calls() else [])
    if not all(os.path.exists(p) for p in made):
        return False
    t = min(os.path.getmtime(p) for p in made)
    return all(os.path.getmtime(p) <= t for p in _deps() + [os.path.abspath(__file__)])


def _compile(src: str, extra) -> str:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc(), "-c", src, "-o", obj] + CFLAGS + list(extra)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        calls = ex.submit(_build_calls) if can_build_calls() else None
        objs = list(ex.map(lambda s: _compile(s, extra), srcs))
        if calls is not None:
            calls.result()
    tmp = LIB + ".tmp"
    cmd = [nvcc(), "-shared", "-o", tmp] + objs + ARCH + ["-cudart", "shared"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
