"""Build libkvsel.so in-tree with nvcc for sm_103a (GB300).

Each .cu file compiles to an object in parallel, then nvcc links them into a
shared library with the CUDA runtime linked statically, so the library loads
on a machine without a GPU driver (symbol checks) and uses the driver only
when a call needs the GPU. Beside it g++ compiles _kvsel_torch.so, the Python
module that hands torch tensors to the paged-cache calls (against the headers
and libraries of the installed torch).

    python -m kv_cache_eviction_snapkv_gb300.build [--verbose]
"""

from __future__ import annotations

import concurrent.futures as cf
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
LIB = os.path.join(PKG, "libkvsel.so")
# debug library: the same sources with -DKVSEL_DEBUG (bounds checks on every
# gather and output write, BAD_INDEX instead of an out-of-range access)
BUILD_DEBUG = os.path.join(PKG, "_build_debug")
LIB_DEBUG = os.path.join(PKG, "libkvsel_debug.so")
SOURCES = ["api.cu", "score_tc.cu", "score_generic.cu", "select.cu", "compact.cu",
           "decode.cu", "jacap.cu", "reverse.cu", "paged_api.cu", "paged_append.cu",
           "paged_attention.cu", "paged_compact.cu", "pages_update.cu"]
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(PKG, "_kvsel_torch.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def _compile(src: str, verbose: bool, debug: bool = False) -> str:
    obj = os.path.join(BUILD_DEBUG if debug else BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *ARCH, "-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC",
           *(["-DKVSEL_DEBUG"] if debug else []),
           "-I", INCLUDE, "-I", CSRC, "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{res.stdout}\n{res.stderr}")
    if verbose and res.stderr:
        sys.stderr.write(res.stderr)
    return obj


def _compile_binding() -> None:
    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise RuntimeError("torch is not installed: the Python binding needs it")
    torch_dir = os.path.dirname(spec.origin)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    tmp = BINDING + ".tmp"
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared",
           *(x for d in (INCLUDE, os.path.join(torch_dir, "include"),
                         os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
                         sysconfig.get_paths()["include"], os.path.join(cuda, "include"))
             for x in ("-I", d)),
           BINDING_SRC, "-o", tmp, "-L", os.path.join(torch_dir, "lib"),
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed for binding.cpp:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, BINDING)


def _current(target: str, deps) -> bool:
    return os.path.exists(target) and os.path.getmtime(target) >= max(map(os.path.getmtime, deps))


def build(verbose: bool = False, force: bool = False, debug: bool = False) -> str:
    """Compile every source and link libkvsel.so (debug: libkvsel_debug.so with
    the bounds checks); returns the library path."""
    lib = LIB_DEBUG if debug else LIB
    os.makedirs(BUILD_DEBUG if debug else BUILD, exist_ok=True)
    header = os.path.join(INCLUDE, "kvsel.h")
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != "binding.cpp"] + [header]
    binding = force or not _current(BINDING, [BINDING_SRC, header])
    if not force and _current(lib, deps):
        if binding:
            _compile_binding()
        return lib
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        also = ex.submit(_compile_binding) if binding else None
        objs = list(ex.map(lambda s: _compile(s, verbose, debug), SOURCES))
        if also is not None:
            also.result()
    tmp = lib + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", tmp, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(verbose="--verbose" in sys.argv, force="--force" in sys.argv,
                debug="--debug" in sys.argv))
