"""Builds libgdla.so (sm_100a) and the binding of its paged-cache calls in-tree, with nvcc and g++.

The library is one translation unit (csrc/gdla_lib.cu). cudart is linked
statically and the driver API is reached through cudaGetDriverEntryPoint, so
the .so loads on machines without a GPU driver (its calls then fail with
GDLA_ERR_CUDA). The binding (csrc/gdla_binding.cpp, a CPython extension on
PyTorch's headers) takes the library's functions by address and links against
PyTorch alone.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_PATH = os.path.join(PKG, "libgdla.so")
BINDING_SOURCES = [os.path.join(CSRC, "gdla_binding.cpp"), os.path.join(INCLUDE, "gdla.h")]
SOURCES = ["gdla_lib.cu", "gdla_api.cu", "gdla_prefill.cu", "gdla_prefill_bwd.cu", "gdla_prologue.cu", "gdla_decode.cu", "gdla_decode_noalloc.cu",
           "gdla_decode_latent.cu", "gdla_selftest.cu", "gdla_internal.h", "gdla_ptx.cuh", "gdla_prologue.h",
           "gdla_pair.cuh", "gdla_paged.cuh", "gdla_cache_append.cu", "gdla_decode_paged.cu"]

ARCH_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the GDLA CUDA library cannot be built")


def _inputs():
    files = [os.path.join(CSRC, s) for s in SOURCES] + [os.path.join(INCLUDE, "gdla.h"), __file__]
    return [f for f in files if os.path.exists(f)]


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH):
        return False
    t = os.path.getmtime(LIB_PATH)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def _compile(cmd):
    # the compiler's intermediate files stay inside the repository
    scratch = os.path.join(os.path.dirname(PKG), "_build", "tmp")
    os.makedirs(scratch, exist_ok=True)
    subprocess.check_call(cmd, env={**os.environ, "TMPDIR": scratch})


def binding_path() -> str:
    """The binding of this interpreter and PyTorch: it reads tensors through their C++ ABI, so its name says which
    ones it was compiled against and one made for others is not found, however new it is."""
    import torch
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    return os.path.join(PKG, f"_gdla_binding.torch-{torch.__version__}-cxx11abi{abi}{sysconfig.get_config_var('EXT_SUFFIX')}")


def build_binding(force: bool = False) -> str:
    """Compile csrc/gdla_binding.cpp into _gdla_binding.*.so next to this file."""
    path = binding_path()
    if not force and os.path.exists(path):
        t = os.path.getmtime(path)
        if all(os.path.getmtime(f) <= t for f in [*BINDING_SOURCES, __file__]):
            return path
    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    tmp = path + f".tmp{os.getpid()}"
    _compile(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
              f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
              "-isystem", os.path.join(base, "include"), "-isystem", os.path.join(base, "include/torch/csrc/api/include"),
              "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(cuda, "include"),
              "-o", tmp, BINDING_SOURCES[0], "-L", os.path.join(base, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu",
              "-ltorch", "-ltorch_python"])
    os.replace(tmp, path)
    return path


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile csrc/gdla_lib.cu into libgdla.so next to this file, and the binding beside it."""
    build_binding(force)
    if not force and up_to_date():
        return LIB_PATH
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH_FLAGS, "-O3", "-lineinfo", "-std=c++17", "--shared", "-Xcompiler", "-fPIC",
           "-Xcompiler", "-fvisibility=hidden", "-I", INCLUDE, "-I", CSRC, "-o", tmp,
           os.path.join(CSRC, "gdla_lib.cu")]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    _compile(cmd)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose=True))
