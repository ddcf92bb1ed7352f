"""Build libadaln.so in-tree with nvcc for sm_103a (GB300).

The translation units are compiled in parallel and linked into
``invariant_dit_adaln_gb300/lib/libadaln.so`` (git-ignored).  Flags:
``-gencode arch=compute_103a,code=sm_103a -O3 -lineinfo --fmad=false``; no
fast math, so every floating-point operation rounds as written.

Beside it g++ builds ``lib/adaln_marshal_<Python>_<torch version>.so``, the
Python module that marshals PyTorch tensors for the calls of
include/adaln_ops.h and include/adaln_tune.h.  It is compiled against the running Python and the
installed PyTorch, hence its name.  The library does not need it: where it
cannot be built, build() warns, and only those calls from Python are missing
(they raise).
"""

from __future__ import annotations

import os
import re
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
LIBDIR = os.path.join(PKG, "lib")
LIB = os.path.join(LIBDIR, "libadaln.so")
HEADERS = ("adaln.h", "adaln_ops.h", "adaln_tune.h")
SOURCES = ["api.cu", "out.cu", "proj.cu", "tc_proj.cu", "res.cu", "f32.cu", "noalloc.cu",
           "ops_api.cu", "heads.cu", "embed.cu", "grads.cu", "tune_api.cu", "ckpt.cu", "lora.cu", "lora_tc.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "--fmad=false", "-std=c++17", "-Xcompiler", "-fPIC",
              "-Xptxas", "-warn-spills", f"-I{INCLUDE}", f"-I{CSRC}"]


MARSHAL_SOURCE = os.path.join(CSRC, "marshal.cpp")


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libadaln.so")


def _inputs():
    files = [os.path.join(CSRC, s) for s in SOURCES]
    files += [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    files += [os.path.join(INCLUDE, f) for f in HEADERS]
    return files


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def marshal_path() -> str:
    import torch
    version = re.sub(r"[^0-9A-Za-z]+", "_", torch.__version__)
    return os.path.join(LIBDIR, f"adaln_marshal_{sys.implementation.cache_tag}_{version}.so")


def _marshal_up_to_date() -> bool:
    path = marshal_path()
    if not os.path.exists(path):
        return False
    inputs = [MARSHAL_SOURCE] + [os.path.join(INCLUDE, f) for f in HEADERS]
    return all(os.path.getmtime(f) <= os.path.getmtime(path) for f in inputs)


def build_marshal() -> str:
    """Compile the marshalling module for the installed PyTorch; returns its path.
    Raises where there is no PyTorch with its headers, or no C++ compiler."""
    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    path = marshal_path()
    os.makedirs(LIBDIR, exist_ok=True)
    tmp = path + f".tmp{os.getpid()}"
    libs = os.path.join(base, "lib")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", f"-I{INCLUDE}",
           f"-I{sysconfig.get_paths()['include']}", f"-I{os.path.join(base, 'include')}",
           f"-I{os.path.join(base, 'include', 'torch', 'csrc', 'api', 'include')}", f"-I{os.path.join(cuda, 'include')}",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", MARSHAL_SOURCE, "-o", tmp, f"-L{libs}",
           f"-Wl,-rpath,{libs}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on marshal.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, path)
    return path


def _try_marshal(force: bool):
    """Build the module if it is out of date; the exception if that fails, for
    any reason: no PyTorch, none with CUDA headers, no compiler."""
    try:
        if force or not _marshal_up_to_date():
            if os.path.exists(marshal_path()):
                os.remove(marshal_path())  # never called with headers other than its own
            build_marshal()
    except Exception as e:
        return e
    return None


def build(force: bool = False, verbose: bool = False, extra_flags=(), variant: str | None = None) -> str:
    """Compile and link the library; returns its path.  `variant` names a test
    build with extra flags, linked to lib/<variant>/libadaln.so with objects in
    _build/<variant>/ (the release library is lib/libadaln.so).  Warns if the
    marshalling module cannot be built."""
    lib = LIB if variant is None else os.path.join(LIBDIR, variant, "libadaln.so")
    objdir = BUILD if variant is None else os.path.join(BUILD, variant)
    with ThreadPoolExecutor(max_workers=1) as ex:
        module = ex.submit(_try_marshal, force) if variant is None else None
        if force or not up_to_date(lib):
            _build_library(lib, objdir, extra_flags, verbose)
        failure = module.result() if module is not None else None
    if failure is not None:
        warnings.warn("libadaln.so is built, but not the module behind the Python calls of adaln_ops.h: "
                      f"{type(failure).__name__}: {failure}", RuntimeWarning, stacklevel=2)
    return lib


def _build_library(lib, objdir, extra_flags, verbose) -> None:
    os.makedirs(objdir, exist_ok=True)
    os.makedirs(os.path.dirname(lib), exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(objdir, os.path.splitext(src)[0] + ".o")
        cmd = [cc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stdout + r.stderr

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    logs = "".join(log for _, log in results)
    if verbose and logs.strip():
        print(logs, file=sys.stderr)
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", tmp, *[o for o, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)


# Test build: the first wait of every waiting kernel goes to an mbarrier that
# nothing arrives on, with a 200 us limit (the kernels' time-out path).
WAIT_TEST_FLAGS = ["-DADALN_TEST_WAIT_NEVER_NS=200000"]


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True,
                extra_flags=["-Xptxas", "-v"] if "-v" in sys.argv else []))
