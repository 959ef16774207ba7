"""Build the sm_100a shared library libw4a4.so in-tree with nvcc.

Each CUDA source compiles to an object in parallel; the objects link into one
shared library next to this file.  The CUDA runtime is linked statically, and
the driver's tensor-map encoder is resolved at run time, so the library
needs no libcuda at link time and builds on a machine without a GPU.  The
CPython extension _binding.so (csrc/binding.cpp, plain C++ over PyTorch's
headers) is built beside it with g++.
"""

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libw4a4.so")
BINDING = os.path.join(HERE, "_binding.so")
SOURCES = ["api.cu", "quant.cu", "quant_tc.cu", "gemm.cu", "gemm_legacy.cu", "smallm.cu", "gemv.cu", "noalloc.cu", "lora.cu",
           "w4a16.cu", "qk_rope.cu", "attention.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _nvcc():
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def _flags(extra=()):
    return ["-O3", "-std=c++17", *ARCH, "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
            "-I", INCLUDE, "-I", CSRC, *extra]


def _up_to_date(obj, deps):
    if not os.path.exists(obj):
        return False
    t = os.path.getmtime(obj)
    return all(os.path.getmtime(d) <= t for d in deps)


def built_for():
    """What _binding.so is tied to: it links PyTorch's and Python's internals."""
    import torch
    return f"torch {torch.__version__}, {sys.implementation.cache_tag}"


def _built_for_this(lib):
    """Whether the extension at `lib` was compiled for this PyTorch and Python
    (the text is in it; one for others is not loaded to ask it)."""
    with open(lib, "rb") as f:
        return f"built for <{built_for()}>".encode() in f.read()


def build_binding(force=False):
    """_binding.so: the marshalling of the block entries."""
    import sysconfig

    import torch

    src = os.path.join(CSRC, "binding.cpp")
    if not force and _up_to_date(BINDING, [src, os.path.join(INCLUDE, "w4a4.h")]) and _built_for_this(BINDING):
        return BINDING
    root = os.path.dirname(torch.__file__)
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DBUILT_FOR="built for <{built_for()}>"', "-I", INCLUDE,
           "-isystem", os.path.join(root, "include"),
           "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"],
           "-isystem", os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include"), src, "-o", BINDING,
           "-L", os.path.join(root, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for binding.cpp:\n{r.stdout}\n{r.stderr}")
    return BINDING


def build(verbose=False, force=False, ptxas_verbose=False):
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    headers = [os.path.join(CSRC, h) for h in os.listdir(CSRC) if h.endswith((".cuh", ".h"))]
    headers.append(os.path.join(INCLUDE, "w4a4.h"))
    extra = ["-Xptxas", "-v"] if ptxas_verbose else []

    def compile_one(src):
        path = os.path.join(CSRC, src)
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        if not force and not ptxas_verbose and _up_to_date(obj, [path, *headers]):
            return obj, ""
        cmd = [nvcc, *_flags(extra), "-c", path, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(build_binding, force)
        results = list(ex.map(compile_one, SOURCES))
        binding.result()
    objs = [o for o, _ in results]
    if verbose or ptxas_verbose:
        for _, log in results:
            if log:
                sys.stderr.write(log)
    if force or not _up_to_date(LIB, objs):
        cmd = [nvcc, *ARCH, "-shared", "-o", LIB, *objs, "-cudart", "static"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    return LIB


if __name__ == "__main__":
    build(verbose=True, force="--force" in sys.argv, ptxas_verbose="--ptxas" in sys.argv)
    print(LIB)
