"""Build libgs.so (the CUDA rasterizer behind include/gs.h) for sm_103a, in-tree.

    python -m differentiable_gaussian_splatting_gb300.build [--force]

Each .cu file is compiled in parallel with nvcc, then linked into
``_build/libgs.so`` next to this file (static CUDA runtime, no other
dependency: it builds without torch).  Beside it
``_build/gs_token_binding.so``, the Python binding of the token operators, is
compiled with g++ against torch's and Python's headers where torch is
installed.  The library is rebuilt when a source or header is newer, the
binding also when it was made for another torch or Python.
"""

from __future__ import annotations

import glob
import importlib.metadata
import importlib.util
import json
import os
import shutil
import subprocess
import sys
import sysconfig
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


def _is_newer(target: str, inputs: list[str]) -> bool:
    """Whether target exists and no input is newer."""
    return os.path.exists(target) and all(
        os.path.getmtime(p) <= os.path.getmtime(target) for p in inputs)


def library_up_to_date() -> bool:
    headers = [p for kind in ("*.h", "*.cuh") for p in glob.glob(os.path.join(CSRC, kind))]
    return _is_newer(LIB, sources() + headers + [os.path.join(INCLUDE, "gs.h")])


def _torch_of_binding() -> dict | None:
    """What the binding is made for: the torch and the Python it is loaded beside (None:
    no torch, which nothing can call it without)."""
    spec = importlib.util.find_spec("torch")
    if spec is None or spec.origin is None:
        return None
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        version = ""
    return {"torch": version, "at": spec.origin, "changed": os.path.getmtime(spec.origin),
            "python": sysconfig.get_config_var("EXT_SUFFIX")}


def binding_up_to_date() -> bool:
    if not _is_newer(BINDING, [os.path.join(CSRC, "token_binding.cpp"),
                               os.path.join(INCLUDE, "gs.h")]):
        return False
    try:
        with open(BINDING + ".json") as f:
            return json.load(f) == _torch_of_binding()
    except (OSError, ValueError):
        return False


def up_to_date() -> bool:
    return library_up_to_date() and (binding_up_to_date() or _torch_of_binding() is None)


def _binding_commands(obj: str, tmp: str) -> tuple[list[str], list[str]]:
    """Compile and link commands of the token operators' binding."""
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


def _run(cmd: list[str], what: str, verbose: bool) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed on {what}:\n{r.stderr}")
    if verbose and r.stderr:
        print(r.stderr, file=sys.stderr)


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Compile and link libgs.so; returns its path."""
    if not force and library_up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    srcs = sources()
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in srcs]
    with ThreadPoolExecutor(max_workers=max(1, len(srcs))) as ex:
        list(ex.map(lambda job: _run([cc, *NVCC_FLAGS, "-I", INCLUDE, "-c", job[0], "-o", job[1]],
                                     os.path.basename(job[0]), verbose), zip(srcs, objs)))
    tmp = LIB + f".tmp{os.getpid()}"
    # the library's own name inside it, so that the binding finds it beside itself
    _run([cc, *ARCH, "-shared", "-Xlinker", "-soname=libgs.so", "-o", tmp, *objs], "libgs.so",
         verbose)
    os.replace(tmp, LIB)
    return LIB


def build_binding(force: bool = False, verbose: bool = False, library=build_library) -> str:
    """Compile the token operators' binding and link it against libgs.so, which `library`
    provides; returns its path."""
    if not force and binding_up_to_date():
        return BINDING
    made_for = _torch_of_binding()
    if made_for is None:
        raise RuntimeError("torch not found: the token operators' binding is built against it")
    os.makedirs(BUILD, exist_ok=True)
    tmp = BINDING + f".tmp{os.getpid()}"
    compile_binding, link_binding = _binding_commands(os.path.join(BUILD, "token_binding.o"), tmp)
    _run(compile_binding, "token_binding.cpp", verbose)
    library()
    _run(link_binding, "gs_token_binding.so", verbose)
    os.replace(tmp, BINDING)
    with open(BINDING + ".json", "w") as f:
        json.dump(made_for, f)
    return BINDING


def build(force: bool = False, verbose: bool = False) -> str:
    """Build the library and, where torch is installed, the binding, side by side; a binding that
    fails leaves the library built.  Returns the library's path."""
    with ThreadPoolExecutor(max_workers=2) as ex:
        library = ex.submit(build_library, force, verbose)
        binding = (ex.submit(build_binding, force, verbose, library.result)
                   if _torch_of_binding() is not None else None)
    path = library.result()
    if binding is not None:
        binding.result()
    return path


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
