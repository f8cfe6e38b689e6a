"""Build the sm_100a shared library libbitnest.so in-tree with nvcc, and, where
torch is installed, the package's binding of the serving calls to its tensors
(_binding.*.so) with g++."""
from __future__ import annotations

import glob
import importlib.util
import os
import runpy
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libbitnest.so")
BINDING_SRC = os.path.join(CSRC, "torch_binding.cpp")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC,-O2",
    "--expt-relaxed-constexpr",
]


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
    deps += glob.glob(os.path.join(INCLUDE, "*.h"))
    return any(os.path.getmtime(d) > t for d in deps)


def binding_path(torch_version: str) -> str:
    """The binding's file.  It uses this Python's and this torch's C++ internals,
    so its name has both: one built for others is neither kept nor loaded."""
    return os.path.join(HERE, f"_binding.{sys.implementation.cache_tag}-torch{torch_version}.so")


def build_binding(force: bool = False, verbose: bool = False) -> str | None:
    """Compile csrc/torch_binding.cpp against the torch that is installed (its
    headers and host libraries; it loads them, and the CUDA library, itself).
    None without torch."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        print("torch is not installed: its binding of the serving calls is not built", file=sys.stderr)
        return None
    torch = os.path.dirname(spec.origin)
    binding = binding_path(runpy.run_path(os.path.join(torch, "version.py"))["__version__"])
    deps = [BINDING_SRC, os.path.join(INCLUDE, "bitnest.h")]
    if not force and os.path.exists(binding) and all(
            os.path.getmtime(d) <= os.path.getmtime(binding) for d in deps):
        return binding
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    inc = [INCLUDE, os.path.join(torch, "include"),
           os.path.join(torch, "include/torch/csrc/api/include"), os.path.join(cuda, "include"),
           sysconfig.get_paths()["include"]]
    tmp = binding + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           "-fvisibility=hidden", *("-I" + d for d in inc), BINDING_SRC, "-o", tmp,
           "-L" + os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    if verbose:
        print(" ".join(cmd))
    subprocess.check_call(cmd)
    for old in glob.glob(os.path.join(HERE, "_binding.*so")):  # of other versions
        os.remove(old)
    os.replace(tmp, binding)
    return binding


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    """The library, which needs no torch, then the binding."""
    build_library(force, verbose, extra)
    build_binding(force, verbose)
    return LIB


def build_library(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    if not force and not _stale():
        return LIB
    nvcc = os.environ.get("NVCC", "nvcc")
    objdir = os.path.join(HERE, "_build")
    os.makedirs(objdir, exist_ok=True)
    objs = []
    procs = []
    for src in sources():
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        cmd = [nvcc, *NVCC_FLAGS, *(extra or []), "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd))
        procs.append((subprocess.Popen(cmd), src))
        objs.append(obj)
    failed = [src for p, src in procs if p.wait() != 0]
    if failed:
        raise RuntimeError(f"nvcc failed for {failed}")
    tmp = LIB + ".tmp"
    cmd = [nvcc, "-shared", "-gencode", "arch=compute_100a,code=sm_100a", *objs, "-o", tmp]
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
    print(LIB)
