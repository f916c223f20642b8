"""Build libfp8mlp.so (the C-ABI library) in-tree with nvcc for sm_100a.

    python -m fp8_relu_mlp_b200.build [--force] [--verbose]

Every translation unit is compiled for ``sm_100a`` only, with -lineinfo and
without fast-math (the scale arithmetic relies on IEEE division and sqrt).
Where torch and Python's headers are there, the module _marshal is built beside
it with g++: the argument marshalling of the calls made per layer.  Without it
the Python binding marshals them itself, so a module that cannot be built is a
warning, and a stale one is removed.  The CUDA runtime is linked statically; the driver's tensor-map encoder is
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
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libfp8mlp.so")
# named for this Python alone: torch's version is all that the binding compares
MARSHAL = os.path.join(PKG, "_marshal" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
UNTAGGED = os.path.join(PKG, "_marshal.so")
# what binding.cpp includes, under torch's include folder
TORCH_HEADERS = ("c10/cuda/CUDAFunctions.h", "c10/cuda/CUDAStream.h", "torch/csrc/autograd/python_variable.h",
                 "torch/headeronly/version.h")

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


def _marshal_command(torch: str) -> list[str] | None:
    """How to build the module, but for its output; None where something is missing."""
    cxx = os.environ.get("CXX") or shutil.which("g++")
    python, include, lib = sysconfig.get_paths()["include"], os.path.join(torch, "include"), os.path.join(torch, "lib")
    try:
        cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    except RuntimeError:
        return None
    needed = [os.path.join(include, h) for h in TORCH_HEADERS]
    needed += [os.path.join(python, "Python.h"), os.path.join(cuda, "cuda_runtime_api.h"), os.path.join(lib, "libc10_cuda.so")]
    if not cxx or not all(os.path.exists(f) for f in needed):
        return None
    return [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-I" + include, "-I" + python, "-I" + cuda,
            os.path.join(CSRC, "binding.cpp"), "-L" + lib, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def _remove(path: str):
    if os.path.exists(path):
        os.remove(path)


def build_marshal(force: bool = False, verbose: bool = False) -> str | None:
    """The module's path, or None where it cannot be built."""
    _remove(UNTAGGED)  # any Python would load it
    spec = importlib.util.find_spec("torch")  # found, not imported
    if spec is None or not spec.origin:
        return None
    torch = os.path.dirname(spec.origin)
    stamp = os.path.join(BUILD, "marshal.stamp")
    h = hashlib.sha256()
    for f in (os.path.join(CSRC, "binding.cpp"), __file__, os.path.join(torch, "version.py")):
        with open(f, "rb") as fh:
            h.update(fh.read())
    h.update(MARSHAL.encode())
    if not force and os.path.exists(MARSHAL) and os.path.exists(stamp) and open(stamp).read() == h.hexdigest():
        return MARSHAL
    _remove(MARSHAL)
    cmd = _marshal_command(torch)
    if cmd is None:
        return None
    tmp = MARSHAL + ".tmp"
    cmd += ["-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
        failed = r.stdout + r.stderr if r.returncode != 0 else None
    except OSError as e:
        failed = str(e)
    if failed is not None:
        warnings.warn(f"the argument marshalling stays in Python: {cmd[0]} failed on binding.cpp:\n{failed}")
        return None
    os.replace(tmp, MARSHAL)
    with open(stamp, "w") as fh:
        fh.write(h.hexdigest())
    return MARSHAL


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    os.makedirs(BUILD, exist_ok=True)
    lib = build_library(force, verbose, extra)
    build_marshal(force, verbose)
    return lib


def build_library(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
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
