"""Build in-tree: libpa.so, every CUDA kernel for sm_100a plus the host block
manager, one shared library exposing the C ABI of include/pa.h; and _calls, the
extension module that marshals torch tensors for the shortest calls.

    python -m paged_kv_cache_414_b200.build [--force] [--verbose]
"""
from __future__ import annotations

import importlib.metadata
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libpa.so")
CALLS = os.path.join(PKG, "_calls" + sysconfig.get_config_var("EXT_SUFFIX"))
BUILD_DIR = os.path.join(ROOT, "_build")

CU_SOURCES = ["library.cu"]
CPP_SOURCES = ["block_manager.cpp"]
HEADERS = sorted(f for f in os.listdir(CSRC) if f.endswith((".cuh", ".cu", ".h")))

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-Xptxas", "-v"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _inputs():
    files = [os.path.join(CSRC, f) for f in CU_SOURCES + CPP_SOURCES + HEADERS]
    files += [os.path.join(INCLUDE, "pa.h"), os.path.abspath(__file__)]
    return files


def _newer(out, inputs) -> bool:
    return os.path.exists(out) and all(os.path.getmtime(f) <= os.path.getmtime(out)
                                       for f in inputs)


def up_to_date() -> bool:
    return _newer(LIB, _inputs())


def _torch_version():
    """The installed torch's version, without importing it; None if there is none."""
    try:
        return importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        return None


def build_calls(force: bool = False) -> str | None:
    """The extension module, against the headers of the installed torch; None without torch, which
    the library itself does not need."""
    src = os.path.join(CSRC, "binding.cpp")
    version = _torch_version()
    if version is None:
        return None
    stamp = os.path.join(BUILD_DIR, "_calls.torch")     # the version it was built against
    if os.path.exists(stamp):
        with open(stamp) as f:
            same = f.read() == version
        if same and not force and _newer(CALLS, [src, os.path.join(INCLUDE, "pa.h")]):
            return CALLS
    import torch
    home = os.path.dirname(torch.__file__)
    inc = os.path.join(home, "include")
    lib = os.path.join(home, "lib")
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    tmp = CALLS + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
           "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"],
           "-isystem", os.path.join(cuda, "include"), src, "-o", tmp, "-L", lib,
           "-lc10", "-lc10_cuda", "-ltorch", "-ltorch_cpu", "-ltorch_python", f"-Wl,-rpath,{lib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
    os.replace(tmp, CALLS)
    os.makedirs(BUILD_DIR, exist_ok=True)
    with open(stamp, "w") as f:
        f.write(version)
    return CALLS


def build(force: bool = False, verbose: bool = False) -> str:
    """The library, then the extension module; the library's path."""
    lib = build_library(force, verbose)
    build_calls(force)
    return lib


def build_library(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    nvcc = _nvcc()
    objs = []
    logs = []
    for src in CU_SOURCES:
        obj = os.path.join(BUILD_DIR, src + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c",
               os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        logs.append(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
        objs.append(obj)
    for src in CPP_SOURCES:
        obj = os.path.join(BUILD_DIR, src + ".o")
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-I", INCLUDE, "-c",
               os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        logs.append(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError("g++ failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
        objs.append(obj)
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-Xcompiler", "-fPIC", "--cudart", "static", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
    os.replace(tmp, LIB)
    with open(os.path.join(BUILD_DIR, "ptxas.log"), "w") as f:
        f.write("\n".join(logs))
    if verbose:
        print("\n".join(logs))
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
