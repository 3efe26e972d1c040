"""Build the package's native code, in the package folder.

The verifier's CUDA library:

    nvcc -O3 -std=c++17 -gencode arch=compute_100a,code=sm_100a -lineinfo
         -Xcompiler -fPIC -shared csrc/libspecdec.cu -o libspecdec.so

The CUDA runtime is linked statically, so the library loads next to any
PyTorch build.  No fast-math: the rejection statistics rely on IEEE expf.

The torch binding of the calls around the verify step (_binding.so, from
csrc/binding.cpp): host code only, against the headers of the PyTorch that is
installed, and built again when that is another one.  Without PyTorch only the
library is built, which C programs use alone.
"""
from __future__ import annotations

import glob
import importlib.metadata
import importlib.util
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libspecdec.so")
BINDING = os.path.join(HERE, "_binding.so")
MAIN = os.path.join(HERE, "csrc", "libspecdec.cu")
BINDING_MAIN = os.path.join(HERE, "csrc", "binding.cpp")
HEADER = os.path.join(ROOT, "include", "specdec.h")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def sources():
    return [s for s in sorted(glob.glob(os.path.join(HERE, "csrc", "*"))) if s != BINDING_MAIN] + [HEADER]


def nvcc():
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _newer(target, srcs) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(s) <= t for s in srcs)


def _built_for() -> str:
    """What a binding is good for; it carries this text."""
    try:
        version = importlib.metadata.version("torch")  # without the time its import takes
    except importlib.metadata.PackageNotFoundError:
        from torch import __version__ as version
    return "torch %s, %s" % (version, sysconfig.get_config_var("SOABI"))


def _binding_up_to_date() -> bool:
    if importlib.util.find_spec("torch") is None:
        return True  # none can be built
    if not _newer(BINDING, [BINDING_MAIN, HEADER]):
        return False
    with open(BINDING, "rb") as f:
        return _built_for().encode() + b"\0" in f.read()


def up_to_date() -> bool:
    return _newer(LIB, sources()) and _binding_up_to_date()


def _build_library(verbose: bool) -> None:
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [nvcc(), "-O3", "-std=c++17", *ARCH, "-lineinfo", "-Xcompiler", "-fPIC", "-shared",
           "-cudart", "static", MAIN, "-o", tmp]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)


def _build_binding(verbose: bool) -> None:
    import torch
    base = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    tmp = BINDING + ".tmp%d" % os.getpid()
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI), '-DBUILT_FOR="%s"' % _built_for(),
           "-I", sysconfig.get_paths()["include"], "-isystem", os.path.join(base, "include"),
           "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"), "-isystem", cuda,
           BINDING_MAIN, "-o", tmp, "-L", os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10",
           "-lc10_cuda", "-ldl"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, BINDING)


def build(force: bool = False, verbose: bool = False) -> str:
    if force or not _newer(LIB, sources()):
        _build_library(verbose)
    if importlib.util.find_spec("torch") is None:
        print("PyTorch is not installed: its binding (_binding.so) is not built", file=sys.stderr)
    elif force or not _binding_up_to_date():
        _build_binding(verbose)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
