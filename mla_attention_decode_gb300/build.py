"""Builds libmla_decode.so in-tree with nvcc for sm_103a (no cmake, no torch), and
_mla_cache.so, the compiled argument marshalling of ``cache.py`` (g++, against
the installed torch's headers).

Each .cu translation unit is compiled in parallel, then linked into one shared
library next to this file.  Rebuilds only when a source or header is newer than
the library.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmla_decode.so")
# the trace build (kernel stamps on, see mla_decode_set_trace), built on request only
BUILD_TRACE = os.path.join(PKG, "_build_trace")
LIB_TRACE = os.path.join(PKG, "libmla_decode_trace.so")
EXT_SRC = os.path.join(CSRC, "mla_cache_ext.cpp")
EXT = os.path.join(PKG, "_mla_cache.so")
EXT_TORCH = os.path.join(BUILD, "ext_torch_version")  # the torch that it was built for
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              f"-I{INCLUDE}", f"-I{CSRC}"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmla_decode.so")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src: str, verbose: bool, out_dir: str = BUILD, defines: tuple = ()) -> str:
    obj = os.path.join(out_dir, os.path.basename(src) + ".o")
    cmd = [_nvcc(), *ARCH, *NVCC_FLAGS, *defines, "-c", src, "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    if verbose and r.stderr:
        print(r.stderr)
    return obj


def _ext_stale() -> bool:
    """Older than its sources, or built for another torch (a file beside it says which)."""
    import torch
    deps = [EXT_SRC, os.path.join(INCLUDE, "mla_cache.h"), os.path.join(INCLUDE, "mla_decode.h")]
    if not os.path.exists(EXT) or any(os.path.getmtime(d) > os.path.getmtime(EXT) for d in deps):
        return True
    return not os.path.exists(EXT_TORCH) or open(EXT_TORCH).read() != str(torch.__version__)


def build_ext() -> str:
    """Compile the Python extension; returns its path."""
    import torch
    os.makedirs(BUILD, exist_ok=True)
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    tmp = EXT + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-std=c++17", "-O2", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DMLA_TORCH_VERSION="{torch.__version__}"', f"-I{INCLUDE}",
           f"-I{os.path.join(root, 'include')}", f"-I{os.path.join(root, 'include', 'torch', 'csrc', 'api', 'include')}",
           f"-I{os.path.join(cuda, 'include')}", f"-I{sysconfig.get_paths()['include']}", EXT_SRC, "-o", tmp,
           f"-L{os.path.join(root, 'lib')}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {os.path.basename(EXT_SRC)}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, EXT)
    with open(EXT_TORCH, "w") as f:
        f.write(str(torch.__version__))
    return EXT


def build(force: bool = False, verbose: bool = False, trace: bool = False) -> str:
    """Compile and link the library (and the Python extension) if needed; returns
    the library's path.  trace=True builds the separate trace library (kernel
    stamps compiled in)."""
    lib, out_dir = (LIB_TRACE, BUILD_TRACE) if trace else (LIB, BUILD)
    defines = ("-DMLA_TRACE=1",) if trace else ()
    ext = not trace and (force or _ext_stale())
    if not force and not _stale(lib):
        if ext:
            build_ext()
        return lib
    os.makedirs(out_dir, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        extension = ex.submit(build_ext) if ext else None
        objs = list(ex.map(lambda s: _compile(s, verbose, out_dir, defines), sources()))
        if extension is not None:
            extension.result()
    tmp = lib + f".tmp{os.getpid()}"
    r = subprocess.run([_nvcc(), *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, trace="--trace" in sys.argv))
