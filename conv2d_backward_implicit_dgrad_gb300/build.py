"""Build libdgrad_gb300.so in-tree with nvcc for sm_103a (``build``), and the
Python module that calls its sequence operators (``bind/``) with g++ against
PyTorch (``build_bind``).  The library needs neither PyTorch nor that module.

Each translation unit under ``csrc/`` is compiled in parallel, then linked
into one shared library with the CUDA runtime linked statically (so loading
it needs no CUDA runtime library on the path).  Run as
``python -m conv2d_backward_implicit_dgrad_gb300.build``.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libdgrad_gb300.so")
BIND_SRC = os.path.join(PKG, "bind", "seq_bind.cpp")
BIND = os.path.join(BUILD, "_seq_bind.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O3", "-I", INCLUDE, "-I", CSRC,
          "--expt-relaxed-constexpr"]


def nvcc() -> str:
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libdgrad_gb300")
    return exe


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _deps():
    return sources() + sorted(glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                              + glob.glob(os.path.join(INCLUDE, "*.h"))) + [__file__]


def up_to_date() -> bool:
    """Whether the library is there and newer than its sources."""
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(d) <= t for d in _deps())


def _run(cmd, what, verbose=False):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{res.stdout}\n{res.stderr}")
    if verbose and (res.stdout or res.stderr):
        print(res.stdout + res.stderr, flush=True)


def build(force: bool = False, verbose: bool = False, extra_flags=(), out: str | None = None) -> str:
    """Compile and link the library; `extra_flags` (e.g. -DDGRAD_TRACE) builds a variant into `out`."""
    if out is None and not force and not extra_flags and up_to_date():
        return LIB
    lib = out or LIB
    objdir = os.path.join(BUILD, "obj" if out is None else "obj_" + os.path.basename(out).replace(".", "_"))
    os.makedirs(objdir, exist_ok=True)
    exe = nvcc()

    def compile_one(src):
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        _run([exe, *ARCH, *CFLAGS, *extra_flags, "-c", src, "-o", obj], f"nvcc on {os.path.basename(src)}", verbose)
        return obj

    # the largest translation units first
    todo = sorted(sources(), key=lambda f: not os.path.basename(f).startswith("seq_scan"))
    with cf.ThreadPoolExecutor(max_workers=min(16, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, todo))
    tmp = lib + f".{os.getpid()}.tmp"
    _run([exe, *ARCH, "-shared", "-cudart", "static", "-Xlinker", "-soname=" + os.path.basename(lib), "-o", tmp, *objs],
         "linking " + os.path.basename(lib))
    os.replace(tmp, lib)
    return lib


# ------------------------------------------------------------ the call module
def _torch_dir() -> str:
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        raise RuntimeError("PyTorch not found: the call module of the sequence operators needs its headers")
    return spec.submodule_search_locations[0]


def _bind_key() -> str:
    """What the call module is built for: it links against PyTorch's C++ interface, which changes with the version."""
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        return f"{sys.implementation.cache_tag}\n{f.read()}"


def bind_fits() -> bool:
    """Whether a call module is there that was built for this Python and PyTorch."""
    try:
        with open(BIND + ".for") as f:
            return os.path.exists(BIND) and f.read() == _bind_key()
    except (OSError, RuntimeError):
        return False


def bind_up_to_date() -> bool:
    if not bind_fits():
        return False
    t = os.path.getmtime(BIND)
    return all(os.path.getmtime(d) <= t for d in (BIND_SRC, os.path.join(INCLUDE, "seq.h"), os.path.join(INCLUDE, "dgrad.h"),
                                                  __file__))


def _compile_bind(obj: str) -> str:
    torch = _torch_dir()
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    system = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
              sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    os.makedirs(os.path.dirname(obj), exist_ok=True)
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-I", INCLUDE, *[a for d in system for a in ("-isystem", d)],
          "-c", BIND_SRC, "-o", obj], "g++ on " + os.path.basename(BIND_SRC))
    return obj


def _link_bind(obj: str) -> str:
    tmp = BIND + f".{os.getpid()}.tmp"
    _run(["g++", "-shared", "-o", tmp, obj, LIB, "-Wl,-rpath,$ORIGIN", "-L" + os.path.join(_torch_dir(), "lib"),
          "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"], "linking " + os.path.basename(BIND))
    if os.path.exists(BIND + ".for"):
        os.remove(BIND + ".for")
    os.replace(tmp, BIND)
    with open(BIND + ".for", "w") as f:
        f.write(_bind_key())
    return BIND


def build_bind(force: bool = False) -> str:
    """Build the call module against the library that is there."""
    if not force and bind_up_to_date():
        return BIND
    return _link_bind(_compile_bind(os.path.join(BUILD, "obj", "seq_bind.o")))


def build_all(force: bool = False, verbose: bool = False) -> str:
    """The library and the call module, compiled side by side.  The library is linked first and stands, whatever
    becomes of the call module."""
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        bind = None
        if force or not bind_up_to_date():
            bind = ex.submit(_compile_bind, os.path.join(BUILD, "obj", "seq_bind.o"))
        build(force=force, verbose=verbose)
        if bind is not None:
            _link_bind(bind.result())
    return LIB


if __name__ == "__main__":
    print(build_all(force="--force" in sys.argv, verbose="-v" in sys.argv))
