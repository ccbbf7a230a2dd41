"""Build libgptq.so in-tree for sm_100a with nvcc (no torch involved), and,
where torch is installed, _serving.so, the CPython module behind serving.py's
allocating calls, with g++ against torch's headers.

    python post_weight_quantization_13_b200/build.py [--force]

(run as a file, not as a module of the package: importing the package loads
the library this script builds)

Objects go to ``post_weight_quantization_13_b200/_build/``; the shared
libraries land next to this file.  Translation units compile in parallel and
are rebuilt only when a source or header is newer than the library, _serving.so
also when it was built for another torch or Python.
"""
from __future__ import annotations

import glob
import os
import importlib.metadata
import importlib.util
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libgptq.so")
EXT = os.path.join(HERE, "_serving.so")
EXT_FOR = os.path.join(BUILD, "_serving.for")   # the torch and Python _serving.so was built for
EXT_SOURCE = os.path.join(CSRC, "serving_ext.cpp")
INCLUDE = os.path.join(ROOT, "include")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O3",
         "--expt-relaxed-constexpr", "-I", INCLUDE]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def _newer(target, inputs) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(p) <= os.path.getmtime(target) for p in inputs)


def up_to_date() -> bool:
    return _newer(LIB, _inputs())


def has_torch() -> bool:
    return importlib.util.find_spec("torch") is not None


def _ext_for() -> str:
    try:
        torch = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:     # on the path, but not installed as a package
        torch = importlib.util.find_spec("torch").origin
    return f"torch {torch}, {sysconfig.get_config_var('SOABI')}"


def ext_up_to_date() -> bool:
    if not _newer(EXT, [EXT_SOURCE, os.path.abspath(__file__)] + glob.glob(os.path.join(INCLUDE, "*.h"))):
        return False
    try:
        with open(EXT_FOR) as f:
            return f.read() == _ext_for()
    except FileNotFoundError:
        return False


def build_ext(verbose: bool = False) -> str:
    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    tmp = EXT + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", INCLUDE, "-isystem", os.path.join(base, "include"),
           "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"), "-isystem", sysconfig.get_paths()["include"],
           EXT_SOURCE, "-o", tmp, LIB, "-Wl,-rpath,$ORIGIN", "-L", os.path.join(base, "lib"),
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {EXT_SOURCE}:\n{r.stdout}\n{r.stderr}")
    if verbose:
        sys.stderr.write(r.stderr)
    os.replace(tmp, EXT)
    os.makedirs(BUILD, exist_ok=True)
    with open(EXT_FOR, "w") as f:
        f.write(_ext_for())
    return EXT


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    if force or not up_to_date():
        _build_lib(verbose, ptxas_info)
    if not has_torch():
        sys.stderr.write("torch is not installed: the 8-bit serving calls of the Python package are not built\n")
    elif force or not ext_up_to_date():
        build_ext(verbose)
    return LIB


def _build_lib(verbose: bool, ptxas_info: bool) -> None:
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [cc, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose or ptxas_info:
            sys.stderr.write(r.stderr)
        return obj

    with ThreadPoolExecutor(max(1, min(8, os.cpu_count() or 1))) as ex:
        objs = list(ex.map(compile_one, sources()))
    tmp = LIB + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-Xlinker", "-soname=libgptq.so", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    force = "--force" in sys.argv
    print(build(force=force, verbose="-v" in sys.argv, ptxas_info="--ptxas" in sys.argv))
