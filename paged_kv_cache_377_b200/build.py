"""Builds libpagedkv.so in-tree with nvcc for sm_100a, and beside it _marshal.so
(csrc/marshal.cpp: the Python side of the small calls, against torch's headers).

``python -m paged_kv_cache_377_b200.build``, or ``build()`` and
``build_marshal()``; each translation
unit of the library compiles in parallel into ``_build/`` and is linked into
``paged_kv_cache_377_b200/libpagedkv.so`` (CUDA runtime linked statically).
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
from typing import List

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libpagedkv.so")
MARSHAL = os.path.join(PKG, "_marshal.so")
MARSHAL_ABI = os.path.join(PKG, "_marshal.abi")  # what it was built for
SOURCES = ["api.cu", "decode.cu", "append.cu", "selftest.cu", "block_manager.cu", "prefill.cu", "prefill_tc.cu",
           "tree.cu", "tables.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
                "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpagedkv.so")


MARSHAL_SOURCE = os.path.join(CSRC, "marshal.cpp")


def _older(built: str, inputs: List[str]) -> bool:
    if not os.path.exists(built):
        return True
    t = os.path.getmtime(built)
    return any(os.path.getmtime(f) > t for f in inputs)


def is_stale() -> bool:
    """Whether libpagedkv.so is missing or older than its sources."""
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, "pagedkv.h"), __file__]
    return _older(LIB, [f for f in files if os.path.isfile(f) and f != MARSHAL_SOURCE])


def _marshal_abi() -> str:
    """What _marshal.so unpacks tensors by: it only serves the torch and the Python it was built for."""
    import sysconfig

    import torch
    return f"torch {torch.__version__} {sysconfig.get_config_var('SOABI')} cxx11 {int(torch.compiled_with_cxx11_abi())}"


def marshal_is_stale() -> bool:
    """Whether _marshal.so is missing, older than its sources, or built for another torch or Python."""
    if _older(MARSHAL, [MARSHAL_SOURCE, os.path.join(INCLUDE, "pagedkv.h"), __file__]):
        return True
    try:
        with open(MARSHAL_ABI) as f:
            return f.read() != _marshal_abi()
    except OSError:
        return True


def _run(cmd: List[str], what: str) -> subprocess.CompletedProcess:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return r


def build(force: bool = False, verbose: bool = False, extra_flags: List[str] = ()) -> str:
    """Compiles and links libpagedkv.so where it is stale. Needs nvcc alone: neither torch nor Python's headers."""
    if not force and not is_stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        r = _run([cc, *FLAGS, *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj], f"nvcc failed on {src}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, file=sys.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    _run([cc, *ARCH, "-shared", "-Xlinker", "-soname,libpagedkv.so", "-o", tmp, *objs], "link failed")
    os.replace(tmp, LIB)
    return LIB


def build_marshal(force: bool = False) -> str:
    """Compiles and links _marshal.so where it is stale, against torch and libpagedkv.so, which has to be there. Apart
    from the library, so that its failure takes nothing from the calls that do without it."""
    if not force and not marshal_is_stale():
        return MARSHAL
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    os.makedirs(BUILD, exist_ok=True)
    abi, obj, gxx = _marshal_abi(), os.path.join(BUILD, "marshal.o"), shutil.which("g++") or "g++"
    include = [a for d in [INCLUDE, *cpp_extension.include_paths(), os.path.join(os.path.dirname(nvcc()), "..", "include"),
                           sysconfig.get_path("include")] for a in ("-I", d)]
    _run([gxx, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", *include, "-c", MARSHAL_SOURCE, "-o", obj],
         "g++ failed on marshal.cpp")
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = MARSHAL + f".tmp{os.getpid()}"
    _run([gxx, "-shared", "-o", tmp, obj, LIB, "-L", lib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10",
          "-lc10_cuda", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"], "link of _marshal.so failed")
    os.replace(tmp, MARSHAL)
    with open(MARSHAL_ABI, "w") as f:
        f.write(abi)
    return MARSHAL


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True,
                extra_flags=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else []))
    print(build_marshal(force="--force" in sys.argv))
