"""Build libds4moe.so (the C ABI of include/ds4moe.h) for sm_100a with nvcc, in-tree, and the Python binding's
short way to some of its calls (csrc/fastcall.cpp), against torch's headers."""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libds4moe.so")
FAST_SRC = os.path.join(CSRC, "fastcall.cpp")
NVCC_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3", "-std=c++17",
              "-Xcompiler", "-fPIC", "-shared"]


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps() -> list[str]:
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + [os.path.join(ROOT, "include", "ds4moe.h"),
                                                                __file__]


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(p) > t for p in _deps())


def fast_path() -> str:
    """Of the Python and the torch that it is built against, so that no other's is loaded."""
    import torch

    return os.path.join(PKG, "_fastcall.%s-torch%s.so" % (sys.implementation.cache_tag, torch.__version__))


def build_fast(force: bool = False) -> str | None:
    """The file at fast_path(); None (and no such file) where it cannot be built: the binding then checks in Python."""
    header = os.path.join(ROOT, "include", "ds4moe.h")
    fast = fast_path()
    if not force and os.path.exists(fast) and os.path.getmtime(fast) >= max(map(os.path.getmtime, (FAST_SRC, header, __file__))):
        return fast
    tmp = fast + ".tmp%d" % os.getpid()
    try:
        import torch
        from torch.utils import cpp_extension

        cuda = os.path.dirname(os.path.dirname(os.path.realpath(subprocess.check_output(
            ["which", os.environ.get("NVCC", "nvcc")], text=True).strip())))
        includes = [*cpp_extension.include_paths(), sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
        libs = os.path.join(os.path.dirname(torch.__file__), "lib")
        subprocess.check_call(["g++", "-O2", "-std=c++20", "-fPIC", "-shared",
                               "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch.compiled_with_cxx11_abi()),
                               *["-I" + i for i in includes], FAST_SRC, "-o", tmp, "-L" + libs, "-ltorch_python", "-ltorch",
                               "-ltorch_cpu", "-lc10", "-lc10_cuda", "-L" + PKG, "-l:libds4moe.so", "-Wl,-rpath,$ORIGIN"])
        os.replace(tmp, fast)
    except (OSError, ImportError, subprocess.CalledProcessError) as e:
        print("%s was not built: %s" % (os.path.basename(fast), e))
        for p in (tmp, fast):
            if os.path.exists(p):
                os.remove(p)
        return None
    return fast


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    _build_lib(force, verbose, extra)
    build_fast(force)
    return LIB


def _build_lib(force: bool, verbose: bool, extra: list[str] | None) -> str:
    if not force and not stale():
        return LIB
    nvcc = os.environ.get("NVCC", "nvcc")
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [nvcc, *NVCC_FLAGS, *(extra or []), "-I", os.path.join(ROOT, "include"), "-o", tmp, *sources()]
    if verbose:
        print(" ".join(cmd))
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    import sys

    print(build(force=True, verbose=True, extra=sys.argv[1:]))
