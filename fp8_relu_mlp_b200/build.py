"""Build libfp8mlp.so (the C-ABI library) in-tree with nvcc for sm_100a.

    python -m fp8_relu_mlp_b200.build [--force] [--verbose]

Every translation unit is compiled for ``sm_100a`` only, with -lineinfo and
without fast-math (the scale arithmetic relies on IEEE division and sqrt).
Where torch and Python's headers are there, _marshal.so is built beside it
with g++: the argument marshalling of the calls made per layer (without it
the Python binding marshals them itself).  The CUDA runtime is linked statically; the driver's tensor-map encoder is
reached through the runtime's driver entry-point query, so the library needs
no libcuda at link time and can be loaded on a machine without a GPU.
"""
from __future__ import annotations

import argparse
import glob
import hashlib
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libfp8mlp.so")
MARSHAL = os.path.join(PKG, "_marshal.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O3", "--expt-relaxed-constexpr",
         "-I" + INCLUDE, "-I" + CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("CUDA_HOME", ""), "/usr/local/cuda"):
        p = os.path.join(cand, "bin", "nvcc") if cand else ""
        if p and os.path.exists(p):
            return p
    p = shutil.which("nvcc")
    if not p:
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libfp8mlp.so")
    return p


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _digest() -> str:
    h = hashlib.sha256()
    for f in sorted(glob.glob(os.path.join(CSRC, "*")) + [os.path.join(INCLUDE, "fp8mlp.h"), __file__]):
        h.update(os.path.basename(f).encode())
        with open(f, "rb") as fh:
            h.update(fh.read())
    h.update(" ".join(ARCH + FLAGS).encode())
    return h.hexdigest()[:16]


def build_marshal(force: bool = False, verbose: bool = False) -> str | None:
    """_marshal.so, or None without torch, its headers, Python's or g++."""
    spec = importlib.util.find_spec("torch")  # found, not imported
    cxx = os.environ.get("CXX") or shutil.which("g++")
    python = sysconfig.get_paths()["include"]
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    if spec is None or not cxx or not os.path.exists(os.path.join(python, "Python.h")):
        return None
    torch = os.path.dirname(spec.origin)
    header = os.path.join(torch, "include", "torch", "csrc", "autograd", "python_variable.h")
    if not os.path.exists(header) or not os.path.exists(os.path.join(torch, "lib", "libc10_cuda.so")):
        return None
    src = os.path.join(CSRC, "binding.cpp")
    stamp = os.path.join(BUILD, "marshal.stamp")
    h = hashlib.sha256()
    for f in (src, __file__, os.path.join(torch, "version.py")):
        with open(f, "rb") as fh:
            h.update(fh.read())
    h.update(" ".join((cxx, python, cuda, torch)).encode())
    if not force and os.path.exists(MARSHAL) and os.path.exists(stamp) and open(stamp).read() == h.hexdigest():
        return MARSHAL
    tmp = MARSHAL + ".tmp"
    lib = os.path.join(torch, "lib")
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-I" + os.path.join(torch, "include"), "-I" + python, "-I" + cuda,
           src, "-o", tmp, "-L" + lib, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {src}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, MARSHAL)
    with open(stamp, "w") as fh:
        fh.write(h.hexdigest())
    return MARSHAL


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    os.makedirs(BUILD, exist_ok=True)
    build_marshal(force, verbose)
    stamp = os.path.join(BUILD, "libfp8mlp.stamp")
    dg = _digest()
    if not force and os.path.exists(LIB) and os.path.exists(stamp) and open(stamp).read() == dg:
        return LIB
    cc = nvcc()
    objs = []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [cc, *ARCH, *FLAGS, *(extra or []), "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)
        return obj

    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, _sources()))
    tmp = LIB + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static", "-lrt", "-ldl", "-lpthread"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    with open(stamp, "w") as fh:
        fh.write(dg)
    return LIB


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-verbose", action="store_true", help="print registers / spills / smem per kernel")
    a = ap.parse_args(argv)
    extra = ["-Xptxas", "-v"] if a.ptxas_verbose else None
    print(build(force=a.force or a.ptxas_verbose, verbose=a.verbose or a.ptxas_verbose, extra=extra))


if __name__ == "__main__":
    sys.exit(main())
