"""Compile the CUDA library in-tree for sm_103a.

Each .cu file under csrc/ is compiled by its own nvcc process (in parallel)
and linked into ``libattn_sm103.so`` next to this file.  nvcc cross-compiles,
so this runs on a machine without a GPU.  csrc/binding.cpp becomes an
extension module (host compiler, PyTorch's headers), for one Python and one
PyTorch: its file's name has both.  The library does not need it.
"""

from __future__ import annotations

import concurrent.futures as cf
import contextlib
import glob
import os
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libattn_sm103.so")
BUILD = os.path.join(HERE, "_build")
# Debug variant: the same sources with -DATTN_DEBUG (explicit bounds checks on
# tensor-copy coordinates and store indices that record a device status
# instead of trapping), built next to the release library.
DEBUG_LIB = os.path.join(HERE, "libattn_sm103_debug.so")
DEBUG_BUILD = os.path.join(HERE, "_build_debug")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", os.path.join(ROOT, "include")]


def _nvcc():
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if c and (os.path.exists(c) or c == "nvcc"):
            return c
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(
        os.path.join(CSRC, "*.h")) + [os.path.join(ROOT, "include", "attn.h"), __file__]


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(p) <= t for p in _deps())


# The extension module of the paged calls; it does not depend on which variant
# of the library is loaded.
BINDING_SRC = os.path.join(CSRC, "binding.cpp")


def binding_path() -> str:
    """The extension module's file for this Python and PyTorch: one that was built
    for others has another name, and is neither loaded nor taken for current."""
    import torch
    abi = sysconfig.get_config_var("SOABI") or sys.implementation.cache_tag
    return os.path.join(HERE, f"_binding.{abi}.torch-{torch.__version__}.so")


def build_binding(force: bool = False) -> str:
    """Compile the extension module with the host compiler."""
    path = binding_path()
    deps = (BINDING_SRC, os.path.join(ROOT, "include", "attn.h"), __file__)
    if not force and os.path.exists(path) and all(os.path.getmtime(p) <= os.path.getmtime(path) for p in deps):
        return path
    import torch
    t = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(_nvcc())) or "/usr/local/cuda"
    tmp = path + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(t, "include"),
           "-I", os.path.join(t, "include", "torch", "csrc", "api", "include"), "-I", os.path.join(cuda, "include"),
           BINDING_SRC, "-o", tmp, "-L", os.path.join(t, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed on {BINDING_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, path)
    return path


def _try_binding(force: bool = False) -> None:
    """The module where the host can build it; a warning where it cannot (no headers
    of Python's or PyTorch's, say): the paged calls then make their checks in Python.
    A module of older sources goes: it would call the new library by the old header."""
    try:
        build_binding(force)
    except Exception as e:
        with contextlib.suppress(ImportError, FileNotFoundError):
            os.remove(binding_path())
        warnings.warn(f"the extension module of the paged calls was not built: {e}", RuntimeWarning, stacklevel=3)


def build(force: bool = False, verbose: bool = False, extra_flags=(), debug: bool = False) -> str:
    """Compile and link the library; with debug=True the -DATTN_DEBUG variant."""
    lib, bdir = (DEBUG_LIB, DEBUG_BUILD) if debug else (LIB, BUILD)
    if debug:
        extra_flags = tuple(extra_flags) + ("-DATTN_DEBUG",)
    if not force and up_to_date(lib):
        _try_binding()
        return lib
    os.makedirs(bdir, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(bdir, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, file=sys.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        binding = ex.submit(_try_binding, force)
        objs = list(ex.map(compile_one, _sources()))
        binding.result()
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, debug="--debug" in sys.argv,
                extra_flags=("-Xptxas", "-v") if "--ptxas-v" in sys.argv else ()))
