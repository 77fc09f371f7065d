"""Build ``libspanla.so`` in-tree with nvcc for sm_103a, and the binding's
extension module ``_fastcall.so`` (csrc/py) with the host compiler.

Each translation unit compiles in parallel into ``_build/``; the objects are
linked into ``hybrid_linear_attention_packed_gb300/libspanla.so`` against the
shared CUDA runtime (the one PyTorch also loads).  Rebuilds only when a source
or header is newer than the library.  The extension module is optional (the
binding makes its calls by ctypes without it): where it cannot be compiled, a
warning says so and the library is built all the same.  It is rebuilt for
another PyTorch or Python, too.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libspanla.so")
EXT_SRC = os.path.join(CSRC, "py", "fastcall.cpp")
EXT = os.path.join(PKG, "_fastcall.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
COMMON = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: libspanla cannot be built")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _headers():
    return (glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
            + glob.glob(os.path.join(INCLUDE, "*.h")))


def _newer(product: str, sources) -> bool:
    if not os.path.exists(product):
        return True
    t = os.path.getmtime(product)
    return any(os.path.getmtime(p) > t for p in sources)


def _stale() -> bool:
    return _newer(LIB, _sources() + _headers() + [__file__])


def _ext_abi() -> str:
    """What the extension module is compiled against: torch and the interpreter."""
    import torch
    return "%s %s" % (torch.__version__, sysconfig.get_config_var("SOABI"))


def _ext_stamp() -> str:
    return os.path.join(BUILD, os.path.basename(EXT) + ".abi")


def _ext_stale() -> bool:
    if _newer(EXT, [EXT_SRC, __file__] + glob.glob(os.path.join(INCLUDE, "*.h"))):
        return True
    try:
        with open(_ext_stamp()) as f:
            return f.read() != _ext_abi()
    except (OSError, ImportError):
        return True


def _compile_ext() -> str:
    """The binding's extension module, against the headers of the torch that is installed."""
    import torch
    tdir = os.path.dirname(torch.__file__)
    cuda_home = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    tmp = EXT + ".tmp.%d" % os.getpid()
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-I", INCLUDE,
           "-I", os.path.join(tdir, "include"), "-I", os.path.join(tdir, "include", "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda_home, "include"),
           "-DSPANLA_TORCH_VERSION=\"%s\"" % torch.__version__, EXT_SRC, "-o", tmp,
           "-L", os.path.join(tdir, "lib"), "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("%s failed on %s:\n%s%s" % (cmd[0], EXT_SRC, r.stdout, r.stderr))
    return tmp


def _install_ext(pending) -> None:
    """Put the compiled module in its place, or warn that there is none (an older one could hold structures of
    another header: it goes)."""
    try:
        tmp = pending.result()
    except Exception as e:   # noqa: BLE001 (no compiler, no headers, ...)
        if os.path.exists(EXT):
            os.remove(EXT)
        warnings.warn("the extension module was not built, its calls go by ctypes: %s" % e)
        return
    os.replace(tmp, EXT)
    with open(_ext_stamp(), "w") as f:
        f.write(_ext_abi())


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    """Compile and link the library and the extension module where stale; returns the library's path."""
    stale, ext_stale = force or _stale(), force or _ext_stale()
    if not stale and not ext_stale:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    extra = ["-Xptxas", "-v"] if ptxas_verbose else []

    def compile_one(src: str):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [_nvcc()] + ARCH + COMMON + extra + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed on %s:\n%s%s" % (src, r.stdout, r.stderr))
        if verbose or ptxas_verbose:
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        ext = ex.submit(_compile_ext) if ext_stale else None
        if stale:
            objs = list(ex.map(compile_one, _sources()))
            tmp = LIB + ".tmp.%d" % os.getpid()
            cmd = [_nvcc()] + ARCH + ["-shared", "-cudart", "shared", "-o", tmp] + objs + [
                "-Xlinker", "-rpath,/usr/local/cuda/lib64"]
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError("link failed:\n%s%s" % (r.stdout, r.stderr))
            os.replace(tmp, LIB)
        if ext is not None:
            _install_ext(ext)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_verbose="--ptxas-v" in sys.argv)
    print(LIB)
