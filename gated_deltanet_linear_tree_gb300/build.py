"""Build libcanopy.so in-tree with nvcc for sm_103a.

Each .cu under csrc/ compiles to an object in parallel; the objects link into
``libcanopy.so`` next to this file (CUDA runtime linked statically, no torch).
Beside it ``_marshal.so``, the native side of the Python binding's short calls
(marshal.cpp: host code, against torch and Python, without the library).  Where
that cannot be built the library is all the same, and the binding's Python side
makes those calls.  Rebuilds only when a source or header is newer than either,
or ``_marshal.so`` was built for another Python or torch.
"""

from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
ROOT = os.path.dirname(PKG)
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libcanopy.so")
MARSHAL = os.path.join(PKG, "_marshal.so")
MARSHAL_TAG = os.path.join(BUILD, "marshal.tag")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE,
         "--expt-relaxed-constexpr", "-Xptxas", "-warn-spills"]


def _nvcc() -> str:
    p = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(p):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libcanopy")
    return p


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _newer(built: str, deps) -> bool:
    return any(os.path.getmtime(d) > os.path.getmtime(built) for d in deps)


def _stale() -> bool:
    deps = sources() + [d for pattern in (os.path.join(CSRC, "*.cuh"), os.path.join(INCLUDE, "*.h"))
                        for d in glob.glob(pattern)]
    return not os.path.exists(LIB) or _newer(LIB, deps)


def marshal_tag() -> str:
    """What ``_marshal.so`` has to be built for: this Python and this torch."""
    import torch
    return f"python {sysconfig.get_config_var('SOABI')}, torch {torch.__version__}"


def _marshal_stale() -> bool:
    if not os.path.exists(MARSHAL) or not os.path.exists(MARSHAL_TAG):
        return True
    with open(MARSHAL_TAG) as f:
        if f.read() != marshal_tag():
            return True
    return _newer(MARSHAL, [os.path.join(CSRC, "marshal.cpp"), *glob.glob(os.path.join(INCLUDE, "*.h"))])


def _build_marshal(nvcc: str) -> None:
    import torch
    root = os.path.dirname(torch.__file__)
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        raise RuntimeError("g++ not found: it builds the Python binding's native side")
    inc = [sysconfig.get_paths()["include"], os.path.join(root, "include"),
           os.path.join(root, "include", "torch", "csrc", "api", "include"),
           os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")]
    tmp = MARSHAL + ".tmp"
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={abi}",
           f'-DCANOPY_MARSHAL_TAG="{marshal_tag()}"', *[f"-I{d}" for d in inc],
           os.path.join(CSRC, "marshal.cpp"), "-o", tmp, "-L" + os.path.join(root, "lib"),
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on marshal.cpp:\n{r.stderr}")
    os.replace(tmp, MARSHAL)
    with open(MARSHAL_TAG, "w") as f:
        f.write(marshal_tag())


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """Compile and link; returns the library path."""
    library, native = force or _stale(), force or _marshal_stale()
    if not library and not native:
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stderr}")
        if verbose and r.stderr.strip():
            print(r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(12, os.cpu_count() or 2)) as ex:
        marshal = ex.submit(_build_marshal, nvcc) if native else None
        if library:
            objs = list(ex.map(compile_one, sources()))
            tmp = LIB + ".tmp"
            r = subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"link failed:\n{r.stderr}")
            os.replace(tmp, LIB)
        if marshal is not None and marshal.exception() is not None:
            warnings.warn(f"_marshal.so was not built; step, prefill and accept take 10 us more of host time a call "
                          f"without it: {marshal.exception()}")
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True))
