"""Build libxs_paged.so in-tree with nvcc for sm_103a (GB300).

Each translation unit compiles in parallel; the shared library links the
CUDA runtime dynamically so it shares the process's runtime (and current
device) with PyTorch.
"""
from __future__ import annotations

import importlib.metadata
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
BUILD_DIR = os.path.join(PKG, "_build")
LIB_NAME = "libxs_paged.so"
LIB_PATH = os.path.join(BUILD_DIR, LIB_NAME)
# Python binding (checks tensors, calls the library by entry address): host
# C++ against PyTorch's headers, one for both libraries.  The library needs
# neither; where PyTorch is not installed, it is all that is built.
BIND_PATH = os.path.join(BUILD_DIR, "xs_bind.so")
BIND_SOURCE = "bind.cpp"
# The debug library: the same sources compiled with -DXS_DEBUG_BOUNDS, so every
# computed global-memory index is checked in the kernels (XS_FLAG_BOUNDS; those
# of kv_swap.cu and block_alloc.cu have no checks).
DEBUG_BUILD_DIR = os.path.join(PKG, "_build_debug")
DEBUG_LIB_PATH = os.path.join(DEBUG_BUILD_DIR, "libxs_paged_debug.so")
SOURCES = ["kv_append.cu", "paged_decode.cu", "kv_swap.cu", "block_alloc.cu", "paged_prefill_tc.cu",
           "qk_norm_rope.cu", "kv4_cache.cu", "kv4_decode.cu", "block_share.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libxs_paged")
    return cand


def _deps() -> list[str]:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != BIND_SOURCE]
    files.append(os.path.join(INCLUDE, "xs_paged.h"))
    return files


def _newer(path: str, files: list[str]) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(f) <= os.path.getmtime(path) for f in files)


def _bind_against() -> str | None:
    """What xs_bind.so is built against: this Python and the PyTorch that it
    finds (None: there is none)."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return None
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        version = str(os.path.getmtime(spec.origin))
    return f"{sys.version}\n{version}\n{spec.origin}\n"


def bind_up_to_date() -> bool:
    """Whether xs_bind.so is newer than its sources and was built against the
    installed PyTorch (or there is none to build it against)."""
    against = _bind_against()
    if against is None:
        return True
    if not _newer(BIND_PATH, [os.path.join(CSRC, BIND_SOURCE), os.path.join(INCLUDE, "xs_paged.h")]):
        return False
    try:
        with open(BIND_PATH + ".against") as f:
            return f.read() == against
    except OSError:
        return False


def up_to_date(debug_bounds: bool = False) -> bool:
    if debug_bounds:
        return _newer(DEBUG_LIB_PATH, _deps())
    return _newer(LIB_PATH, _deps()) and bind_up_to_date()


def build_bind() -> str:
    """Build xs_bind.so with the host compiler."""
    import torch

    os.makedirs(BUILD_DIR, exist_ok=True)
    top = os.path.join(torch.__path__[0], "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    tmp = BIND_PATH + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-I", INCLUDE,
           "-I", top, "-I", os.path.join(top, "torch", "csrc", "api", "include"), "-I", cuda,
           "-I", sysconfig.get_paths()["include"], os.path.join(CSRC, BIND_SOURCE), "-o", tmp,
           "-L", os.path.join(torch.__path__[0], "lib"), "-lc10", "-ltorch_cpu", "-lc10_cuda",
           "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {BIND_SOURCE}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BIND_PATH)
    with open(BIND_PATH + ".against", "w") as f:
        f.write(_bind_against() or "")
    return BIND_PATH


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None,
          debug_bounds: bool = False) -> str:
    """Build the release library (or, with debug_bounds, the debug library with
    in-kernel bounds checks) unless it is newer than every source, and with the
    release library the Python binding where PyTorch is installed; returns the
    library's path."""
    build_dir = DEBUG_BUILD_DIR if debug_bounds else BUILD_DIR
    lib_path = DEBUG_LIB_PATH if debug_bounds else LIB_PATH
    if not force and up_to_date(debug_bounds):
        return lib_path
    os.makedirs(build_dir, exist_ok=True)
    flags = ["-O3", "-std=c++17", *ARCH, "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE,
             "-I", CSRC, *(["-DXS_DEBUG_BOUNDS"] if debug_bounds else []), *(extra_flags or [])]
    if verbose:
        flags += ["-Xptxas", "-v"]
    exe = nvcc()

    def compile_one(src: str) -> str:
        obj = os.path.join(build_dir, os.path.splitext(src)[0] + ".o")
        cmd = [exe, *flags, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            sys.stderr.write(r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        bind = None
        if not debug_bounds and _bind_against() is not None and (force or not bind_up_to_date()):
            bind = ex.submit(build_bind)
        if force or not _newer(lib_path, _deps()):
            objs = list(ex.map(compile_one, SOURCES))
            tmp = lib_path + f".tmp{os.getpid()}"
            cmd = [exe, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs]
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
            os.replace(tmp, lib_path)
        if bind is not None:
            bind.result()       # (after the library is in place: it does not need the binding)
    return lib_path


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                debug_bounds="--debug-bounds" in sys.argv))
