"""Build libcsa2.so (all CUDA sources under csrc/) for sm_100a and _native.so (csrc/binding.cpp, the
torch-side fast path of the calls made per layer), in-tree.

    python -m sparse_attention_fp4_pack_b200.build [--force] [--verbose-ptxas]
"""
import glob
import importlib.metadata
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libcsa2.so")
BINDING = os.path.join(CSRC, "binding.cpp")
NATIVE = os.path.join(HERE, "_native.so")
NATIVE_FOR = os.path.join(HERE, "_native.built_for")  # the Python and torch that _native.so was built for
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    # share the CUDA runtime with the host process (torch), so the current device and
    # streams are the caller's
    "-cudart", "shared",
    "--threads", "4",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in sources() + headers())


def native_for() -> str:
    """What _native.so's binary interface depends on besides its sources."""
    return f"python {sys.version} in {sys.prefix}, torch {importlib.metadata.version('torch')}"


def native_up_to_date() -> bool:
    if not os.path.exists(NATIVE) or not os.path.exists(NATIVE_FOR):
        return False
    with open(NATIVE_FOR) as f:
        if f.read() != native_for():
            return False
    return all(os.path.getmtime(p) <= os.path.getmtime(NATIVE) for p in (BINDING, os.path.join(INCLUDE, "csa2.h")))


def build_native(force: bool = False) -> str:
    """_native.so, linked against libcsa2.so beside it and the installed torch."""
    if not force and native_up_to_date():
        return NATIVE
    from torch.utils import cpp_extension
    cuda = os.path.dirname(os.path.dirname(NVCC))
    dirs = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(cuda, "include"), *cpp_extension.include_paths()]
    libs = cpp_extension.library_paths()
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           *[f"-isystem{d}" for d in dirs], BINDING, "-o", NATIVE + ".tmp", f"-L{HERE}", "-l:libcsa2.so",
           "-Wl,-rpath,$ORIGIN", *[f"-L{d}" for d in libs], *[f"-Wl,-rpath,{d}" for d in libs],
           "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    subprocess.run(cmd, check=True)
    os.replace(NATIVE + ".tmp", NATIVE)
    with open(NATIVE_FOR, "w") as f:
        f.write(native_for())
    return NATIVE


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    build_lib(force, verbose_ptxas)
    build_native(force)
    return LIB


def build_lib(force: bool = False, verbose_ptxas: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    cmd = [NVCC, *FLAGS, "-I", INCLUDE, "-I", CSRC, "-o", LIB + ".tmp", *sources()]
    if verbose_ptxas:
        cmd.insert(1, "-Xptxas=-v")
    subprocess.run(cmd, check=True)
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="--verbose-ptxas" in sys.argv))
