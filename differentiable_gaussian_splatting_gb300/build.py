"""Build libgs.so (the CUDA rasterizer behind include/gs.h) for sm_103a, in-tree.

    python -m differentiable_gaussian_splatting_gb300.build [--force]

Each .cu file is compiled in parallel with nvcc, then linked into
``_build/libgs.so`` next to this file (static CUDA runtime, no other
dependency).  Beside it ``_build/gs_token_binding.so``, the Python binding of
the token operators, is compiled with g++ against torch's headers.  A rebuild
happens when any source or header is newer than the libraries.
"""

from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libgs.so")
BINDING = os.path.join(BUILD, "gs_token_binding.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", *ARCH]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: libgs needs the CUDA toolkit to build")
    return path


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs() -> list[str]:
    return sources() + [p for kind in ("*.h", "*.cuh", "*.cpp")
                        for p in glob.glob(os.path.join(CSRC, kind))] + [
        os.path.join(INCLUDE, "gs.h")]


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(BINDING):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    return all(os.path.getmtime(p) <= t for p in _inputs())


def _binding_commands(obj: str, tmp: str) -> tuple[list[str], list[str]]:
    """Compile and link commands of the token operators' binding."""
    import sysconfig

    import torch

    base = os.path.dirname(torch.__file__)
    lib = os.path.join(base, "lib")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    dirs = [INCLUDE, os.path.join(base, "include"),
            os.path.join(base, "include", "torch", "csrc", "api", "include"),
            os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    cxx = shutil.which("g++") or "c++"
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    return ([cxx, "-O2", "-std=c++17", "-fPIC", "-w", f"-D_GLIBCXX_USE_CXX11_ABI={abi}",
             *[f"-I{d}" for d in dirs], "-c", os.path.join(CSRC, "token_binding.cpp"), "-o", obj],
            [cxx, "-shared", "-o", tmp, obj, LIB, f"-L{lib}", "-ltorch_python", "-ltorch_cpu",
             "-lc10", "-lc10_cuda", f"-Wl,-rpath,{lib}", "-Wl,-rpath,$ORIGIN"])


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link libgs.so; returns its path."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    srcs = sources()
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in srcs]

    def run(cmd, what):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{os.path.basename(cmd[0])} failed on {what}:\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr, file=sys.stderr)

    tmp = LIB + f".tmp{os.getpid()}"
    tmp_binding = BINDING + f".tmp{os.getpid()}"
    binding_obj = os.path.join(BUILD, "token_binding.o")
    compile_binding, link_binding = _binding_commands(binding_obj, tmp_binding)
    jobs = [(compile_binding, "token_binding.cpp")]
    jobs += [([cc, *NVCC_FLAGS, "-I", INCLUDE, "-c", src, "-o", obj], os.path.basename(src))
             for src, obj in zip(srcs, objs)]
    with ThreadPoolExecutor(max_workers=len(jobs)) as ex:
        list(ex.map(lambda job: run(*job), jobs))
    # the library's own name inside it, so that the binding finds it beside itself
    run([cc, *ARCH, "-shared", "-Xlinker", "-soname=libgs.so", "-o", tmp, *objs], "libgs.so")
    os.replace(tmp, LIB)
    run(link_binding, "gs_token_binding.so")
    os.replace(tmp_binding, BINDING)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
