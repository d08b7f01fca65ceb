"""Build step for the CUDA libraries (nvcc, sm_103a only).

Compiles ``csrc/*.cu`` in parallel into ``_build/`` and links
``libmc2_gb300.so`` (the operations) next to this file, ``calib/*.cu``
into ``libmc2_calib.so`` (a measurement probe that only the benchmark loads),
and ``binding/native.cpp`` into ``_native.<python>-torch<version>.so`` (the Python binding's fast calls).
Rebuilds a library only when one of its sources or the public header is newer
than it.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
CALIB = os.path.join(HERE, "calib")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmc2_gb300.so")
CALIB_LIB = os.path.join(HERE, "libmc2_calib.so")
NATIVE_SRC = os.path.join(HERE, "binding", "native.cpp")

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def sources(src_dir=CSRC):
    return sorted(glob.glob(os.path.join(src_dir, "*.cu")))


def _deps(src_dir=CSRC):
    return sources(src_dir) + glob.glob(os.path.join(src_dir, "*.cuh")) + glob.glob(os.path.join(src_dir, "*.h")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h")) + [os.path.abspath(__file__)]


def needs_build(lib=LIB, src_dir=CSRC) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(d) > t for d in _deps(src_dir))


def _build_one(lib, src_dir, force, verbose, extra_flags):
    if not force and not needs_build(lib, src_dir):
        return lib
    os.makedirs(BUILD, exist_ok=True)
    nvcc = NVCC if os.path.exists(NVCC) else "nvcc"
    srcs = sources(src_dir)
    tag = os.path.basename(src_dir)

    def compile_one(src):
        obj = os.path.join(BUILD, f"{tag}_{os.path.basename(src)}.o")
        cmd = [nvcc, *ARCH, *FLAGS, *extra_flags, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)
        return obj

    with ThreadPoolExecutor(max_workers=len(srcs)) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-Xlinker", f"-soname={os.path.basename(lib)}", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Build the operations library (and return its path)."""
    return _build_one(LIB, CSRC, force, verbose, extra_flags)


def native_lib() -> str:
    """Where the binding's extension module is.  It is bound to one Python and one torch, so its name says
    which: after an upgrade of either the old one is not loaded."""
    import torch
    return os.path.join(HERE, f"_native.{sysconfig.get_config_var('SOABI')}-torch{torch.__version__}.so")


def build_native(force: bool = False, verbose: bool = False) -> str:
    """Build the binding's extension module (and return its path)."""
    module = native_lib()
    deps = [NATIVE_SRC, os.path.abspath(__file__)] + glob.glob(os.path.join(ROOT, "include", "*.h"))
    if not force and os.path.exists(module) and all(os.path.getmtime(d) <= os.path.getmtime(module) for d in deps):
        return module
    import torch
    t = os.path.dirname(os.path.abspath(torch.__file__))
    inc = [os.path.join(t, "include"), os.path.join(t, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include"),
           os.path.join(ROOT, "include")]
    lib = os.path.join(t, "lib")
    tmp = module + f".tmp{os.getpid()}"
    # the library of the operations by its name, found beside the module; torch's by theirs
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[f"-I{i}" for i in inc], NATIVE_SRC, "-o", tmp, f"-L{HERE}", "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN",
           f"-L{lib}", f"-Wl,-rpath,{lib}", "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {os.path.basename(NATIVE_SRC)}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, module)
    return module


def build_calib(force: bool = False, verbose: bool = False) -> str:
    """Build the benchmark's calibration probe library (and return its path)."""
    return _build_one(CALIB_LIB, CALIB, force, verbose, ())


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True))
    print(build_native(force="--force" in sys.argv, verbose=True))
    print(build_calib(force="--force" in sys.argv, verbose=True))
