"""Builds libpagedfp8.so in-tree with nvcc for sm_103a (no CMake, no torch
extension machinery): each .cu compiles in parallel, then one shared link.

    python -m paged_fp8_kv_03_gb300.build [--force]
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB_DIR = os.path.join(PKG, "lib")
LIB = os.path.join(LIB_DIR, "libpagedfp8.so")

# The Python binding's fast path.  It holds what it needs of torch's C++ interface, so it serves the
# torch and the Python that it was built with, and says so in its name; without it the same calls are
# checked in Python.
BINDING = os.path.join(LIB_DIR, f"_binding.{sys.implementation.cache_tag}.torch-{torch.__version__}.so")

SOURCES = ["append.cu", "decode.cu", "api.cu", "noalloc.cu", "calibrate.cu", "prefill.cu",
           "rows_fp4.cu", "prefill_fp4.cu", "decode_fp4.cu", "api_fp4.cu",
           "rows_fp8b.cu", "prefill_fp8b.cu", "prefill_direct.cu", "decode_fp8b.cu", "api_fp8b.cu", "pages.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA library cannot be built")
    return cand


def _deps() -> list:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != "binding.cpp"]
    files.append(os.path.join(INCLUDE, "pagedfp8.h"))
    files.append(os.path.abspath(__file__))
    return files


def _binding_deps() -> list:
    return [os.path.join(CSRC, "binding.cpp"), os.path.join(INCLUDE, "pagedfp8.h"), os.path.abspath(__file__)]


def _stale(target: str, files: list) -> bool:
    return not os.path.exists(target) or any(os.path.getmtime(f) > os.path.getmtime(target) for f in files)


def needs_build() -> bool:
    return _stale(LIB, _deps()) or _stale(BINDING, _binding_deps())


def _binding_commands() -> tuple:
    """The commands that compile and link the binding's fast path, and the file they make."""
    base = os.path.dirname(torch.__file__)
    obj, tmp = os.path.join(BUILD, "binding.o"), BINDING + f".tmp{os.getpid()}"
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    cxx = shutil.which("g++") or "c++"
    compile_ = [cxx, "-O2", "-std=c++17", "-fPIC", "-Wall", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                "-I", INCLUDE, "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"),
                "-isystem", os.path.join(base, "include"),
                "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"),
                "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj]
    link = [cxx, "-shared", "-o", tmp, obj, "-L", LIB_DIR, "-lpagedfp8", "-Wl,-rpath,$ORIGIN", "-L",
            os.path.join(base, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    return compile_, link, tmp


def _start(cmd: list):
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)


def _finish(proc, verbose: bool) -> bool:
    out, _ = proc.communicate()
    if verbose or proc.returncode != 0:
        sys.stderr.write(out)
    return proc.returncode == 0


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not needs_build():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    procs = []
    objs = []
    library, binding = force or _stale(LIB, _deps()), force or _stale(BINDING, _binding_deps())
    for src in SOURCES if library else ():
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(obj)
        cmd = [nvcc, *ARCH, *FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        procs.append((src, _start(cmd)))
    if binding:
        compile_, link, binding_tmp = _binding_commands()
        compiled = _start(compile_)
    failed = [src for src, p in procs if not _finish(p, verbose)]
    compiled = binding and _finish(compiled, verbose)
    if failed:
        raise RuntimeError(f"nvcc failed for {failed}")
    if library:
        tmp = LIB + f".tmp{os.getpid()}"
        subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], check=True)
        os.replace(tmp, LIB)
    if compiled and _finish(_start(link), verbose):
        os.replace(binding_tmp, BINDING)
    elif binding:
        sys.stderr.write("the binding's fast path cannot be built here: its calls are checked in Python\n")
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
