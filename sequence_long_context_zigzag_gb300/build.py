"""Build the in-tree CUDA library ``libusp.so`` for sm_103a with nvcc (no cmake, no torch extension).

Each .cu file compiles to an object in parallel (``-gencode arch=compute_103a,code=sm_103a``), then
the objects link into one shared library with the CUDA runtime linked statically, so the library has
no load-time dependency on libcudart or libcuda (driver entry points are fetched at run time).

Beside them the C++ binding of the paged cache's and the rotation's calls (csrc/binding.cpp), a CPython module against the
installed torch, compiles with g++ (a few seconds; its file name carries the torch and Python versions and a
hash of its sources). The library does not depend on it: where it cannot be built (no torch, no Python
headers, no g++), build() warns, and the first call that needs the binding raises.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libusp.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def _nvcc():
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _newest_header():
    hs = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    return max((os.path.getmtime(h) for h in hs), default=0.0)


def _compile(src, obj, extra):
    cmd = [_nvcc(), *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    return r.stderr


def binding_path() -> str:
    """The binding for this interpreter and torch, from the sources as they are now: it takes the ABI's structs by value
    through plain addresses, so one from another usp.h would pass arguments to the wrong places."""
    import hashlib
    import sysconfig

    import torch
    h = hashlib.sha256()
    for src in (BINDING_SRC, os.path.join(INCLUDE, "usp.h")):
        with open(src, "rb") as f:
            h.update(f.read())
    name = f"torch{torch.__version__}_{sysconfig.get_config_var('SOABI')}_{h.hexdigest()[:12]}"
    return os.path.join(PKG, "_usp_binding_" + "".join(c if c.isalnum() else "_" for c in name) + ".so")


def _build_binding(path: str) -> str:
    import inspect
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    def dirs(f):  # the argument's name differs between torch versions
        return f("cuda") if "device_type" in inspect.signature(f).parameters else f(True)
    tmp = f"{path}.{os.getpid()}.tmp"
    cmd = [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", BINDING_SRC, "-o", tmp, "-I", INCLUDE,
           "-I", sysconfig.get_paths()["include"], *[f"-I{d}" for d in dirs(cpp_extension.include_paths)],
           *[f"-L{d}" for d in dirs(cpp_extension.library_paths)], "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for binding.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, path)
    return r.stderr


def build_binding(force: bool = False) -> str:
    path = binding_path()
    if force or not os.path.exists(path):
        _build_binding(path)
    return path


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    hdr_t = _newest_header()
    jobs = []
    objs = []
    for s in srcs:
        o = os.path.join(BUILD, os.path.basename(s)[:-3] + ".o")
        objs.append(o)
        if force or not os.path.exists(o) or os.path.getmtime(o) < max(os.path.getmtime(s), hdr_t):
            jobs.append((s, o))
    with cf.ThreadPoolExecutor(max_workers=1) as ex:  # beside nvcc
        binding = ex.submit(build_binding, force)
        lib = _build_lib(jobs, objs, force, verbose, extra_flags)
        try:
            binding.result()
        except Exception as e:
            warnings.warn(f"the binding of the paged cache's calls was not built: {e}", RuntimeWarning)
    return lib


def _build_lib(jobs, objs, force, verbose, extra_flags) -> str:
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 4)) as ex:
            futs = {ex.submit(_compile, s, o, list(extra_flags)): s for s, o in jobs}
            for f in cf.as_completed(futs):
                msg = f.result()
                if verbose and msg:
                    sys.stderr.write(msg)
    if force or jobs or not os.path.exists(LIB):
        tmp = LIB + ".tmp"
        cmd = [_nvcc(), *ARCH, "-shared", "--cudart", "static", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
