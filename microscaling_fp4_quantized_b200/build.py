"""Build the CUDA library ``libsage_fp4.so`` in-tree for sm_100a with nvcc.

Each ``csrc/*.cu`` is compiled to an object under ``_build/`` and the objects are
linked into a shared library next to this file (CUDA runtime linked statically, so the
library loads on a machine without a GPU driver; the driver API is reached at run time
through cudaGetDriverEntryPoint). ``--checks`` builds the bounds-checked variant
``libsage_fp4_checks.so`` instead (compiled with SAGE_CHECKS: every computed global index
of the quantization and attention kernels is tested before the access; a failure is
reported in the device error word and the access skipped).

    python -m microscaling_fp4_quantized_b200.build [--force] [--verbose] [--checks]

``csrc/binding.cpp``, the native Python binding of the paged cache operators, then becomes the extension
module ``_binding.so`` next to it (g++, torch's headers and libraries; no CUDA code of its own). Without
torch it is left out. It is built again when torch or Python changes: it uses torch's C++ interface,
which is another one in every release.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libsage_fp4.so")
LIB_CHECKS = os.path.join(PKG, "libsage_fp4_checks.so")
BINDING = os.path.join(PKG, "_binding.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
CFLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xptxas", "-v",
                 "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps():
    files = _sources()
    files += [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return files + [os.path.abspath(__file__)]


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(f) <= t for f in _deps())


def build(force: bool = False, verbose: bool = False, checks: bool = False) -> str:
    lib = _build_library(force, verbose, checks)
    build_binding(force)
    return lib


def _build_library(force: bool, verbose: bool, checks: bool) -> str:
    lib = LIB_CHECKS if checks else LIB
    if not force and up_to_date(lib):
        return lib
    bdir = BUILD + ("_checks" if checks else "")
    os.makedirs(bdir, exist_ok=True)
    nvcc = _nvcc()
    flags = CFLAGS + (["-DSAGE_CHECKS"] if checks else [])

    def compile_one(src):
        obj = os.path.join(bdir, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc] + flags + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, r

    objs = []
    with cf.ThreadPoolExecutor(max_workers=4) as ex:
        for src, obj, r in ex.map(compile_one, _sources()):
            if r.returncode != 0:
                sys.stderr.write(r.stdout + r.stderr)
                raise RuntimeError(f"nvcc failed on {src}")
            if verbose:
                sys.stderr.write(r.stderr)
            objs.append(obj)
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [nvcc] + ARCH + ["-shared", "-o", tmp] + objs + ["-lrt", "-ldl", "-lpthread"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("link failed")
    os.replace(tmp, lib)
    return lib


def build_binding(force: bool = False) -> Optional[str]:
    """The binding's path; None without torch."""
    spec = importlib.util.find_spec("torch")
    if spec is None or spec.origin is None:
        sys.stderr.write("torch is not installed: the Python binding is not built\n")
        return None
    src = os.path.join(CSRC, "binding.cpp")
    troot = os.path.dirname(os.path.abspath(spec.origin))
    tlib = os.path.join(troot, "lib")
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           "-I", INCLUDE, "-isystem", os.path.join(troot, "include"),
           "-isystem", os.path.join(troot, "include", "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(cuda, "include"), src,
           "-L", tlib, "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath," + tlib]
    # What the file is good for, kept beside the objects: times alone do not tell.
    built_for = "\n".join([f"torch {importlib.metadata.version('torch')}",
                           f"Python {sysconfig.get_config_var('SOABI')}"] + cmd[1:])
    stamp = os.path.join(BUILD, "binding.txt")
    deps = (src, os.path.join(INCLUDE, "sage_fp4.h"), os.path.abspath(__file__))
    if (not force and os.path.exists(BINDING) and os.path.exists(stamp)
            and all(os.path.getmtime(f) <= os.path.getmtime(BINDING) for f in deps)):
        with open(stamp) as f:
            if f.read() == built_for:
                return BINDING
    import torch
    os.makedirs(BUILD, exist_ok=True)
    tmp = BINDING + f".tmp{os.getpid()}"
    r = subprocess.run(cmd + [f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-o", tmp],
                       capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("the binding did not build")
    os.replace(tmp, BINDING)
    with open(stamp, "w") as f:
        f.write(built_for)
    return BINDING


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--checks", action="store_true", help="the bounds-checked variant")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose, checks=a.checks))
