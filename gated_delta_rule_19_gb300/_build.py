"""Builds libgdn.so in-tree with nvcc for sm_103a (one -gencode, parallel TUs), and _layer.so,
the C++ binding of the linear-attention layer's calls, with g++ against torch's headers."""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libgdn.so")
BINDING = os.path.join(PKG, "_layer.so")
BINDING_SRC = os.path.join(CSRC, "layer_binding.cpp")
BUILD_DIR = os.path.join(PKG, "_build")
BINDING_FOR = os.path.join(BUILD_DIR, "layer_built_for.txt")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC] + ARCH


def nvcc() -> str:
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    cand = os.path.join(cuda, "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(
        os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))


def is_stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(f) > t for f in _deps())


def _built_for() -> str:
    """What the binding is compiled against besides its sources."""
    from importlib import metadata

    try:
        torch = metadata.version("torch")
    except metadata.PackageNotFoundError:
        torch = None
    return f"torch {torch}, Python {sys.version}, {PKG}"


def _binding_is_stale() -> bool:
    try:
        with open(BINDING_FOR) as f:
            if f.read() != _built_for():
                return True
        t = os.path.getmtime(BINDING)
    except OSError:
        return True
    return any(os.path.getmtime(f) > t for f in (BINDING_SRC, os.path.join(INCLUDE, "gdn.h")))


def _binding_dirs() -> list[str]:
    """The folders of torch's, Python's and CUDA's headers; FileNotFoundError if some, or
    torch's CUDA library, are not installed."""
    import sysconfig

    try:
        import torch
        from torch.utils import cpp_extension
    except ImportError as e:
        raise FileNotFoundError(f"no torch: {e}") from e
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    dirs = [*cpp_extension.include_paths(), sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    for header in ("ATen/EmptyTensor.h", "Python.h", "cuda_runtime_api.h"):
        if not any(os.path.exists(os.path.join(d, header)) for d in dirs):
            raise FileNotFoundError(f"{header} is not in any of {dirs}")
    if not os.path.exists(os.path.join(os.path.dirname(torch.__file__), "lib", "libc10_cuda.so")):
        raise FileNotFoundError("torch is installed without CUDA")
    return dirs


def build_binding(verbose: bool = False) -> str | None:
    """Compile the C++ binding against the installed torch.  Without its headers the library
    is all that can be built, and serves every caller of the C ABI: a warning, and no binding
    (gdn.py's calls of the layer then raise)."""
    try:
        dirs = _binding_dirs()
    except FileNotFoundError as e:
        if os.path.exists(BINDING):
            os.remove(BINDING)  # it is of other sources or another torch
        warnings.warn(f"the linear-attention layer's Python binding is not built: {e}", stacklevel=2)
        return None
    import torch

    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", INCLUDE, *(f for d in dirs for f in ("-isystem", d)), BINDING_SRC, "-o", tmp, "-L" + lib,
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-ldl"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {BINDING_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    os.makedirs(BUILD_DIR, exist_ok=True)
    with open(BINDING_FOR, "w") as f:
        f.write(_built_for())
    return BINDING


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile every csrc/*.cu to an object file (in parallel) and link libgdn.so; compile
    the binding beside them."""
    with ThreadPoolExecutor(1) as ex:
        binding = ex.submit(build_binding, verbose) if force or _binding_is_stale() else None
        if force or is_stale():
            _build_lib(verbose, extra_flags)
        if binding is not None:
            binding.result()
    return LIB


def _build_lib(verbose: bool, extra_flags) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs = _sources()
    objs = [os.path.join(BUILD_DIR, os.path.basename(s)[:-3] + ".o") for s in srcs]

    def compile_one(pair):
        src, obj = pair
        cmd = [nvcc(), *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, r

    with ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 4))) as ex:
        results = list(ex.map(compile_one, zip(srcs, objs)))
    for src, r in results:
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, file=sys.stderr)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
