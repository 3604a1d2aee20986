"""Build libfp8q.so (in-tree) from csrc/*.cu for sm_100a with nvcc.

    python -m scaling_aware_transpose_b200.build [--force]

Objects go to _build/ (git-ignored); ptxas register/spill reports to
_build/ptxas.log.  The shared library lands next to this file so that it travels with
the source tree, and beside it _moe_binding.so, the native half of moe.py's helpers
(csrc/moe_binding.cpp: g++ against torch's headers, linked to the library).
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libfp8q.so")
BINDING = os.path.join(PKG, "_moe_binding.so")
BINDING_KEY = os.path.join(BUILD, "moe_binding.key")
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-fmad=false",            # the SwiGLU spec is individually rounded fp32 operations
    "-Xcompiler", "-fPIC",
    "-Xptxas", "-v",
    "-I", INCLUDE, "-I", CSRC,
]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
                  + glob.glob(os.path.join(INCLUDE, "*.h")))


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src):
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    if _stale(obj, [src, *_headers()]):
        r = subprocess.run([NVCC, *FLAGS, "-c", src, "-o", obj], capture_output=True, text=True)
        if r.returncode:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        with open(obj + ".ptxas.txt", "w") as f:
            f.write(r.stderr)
    return obj


def _binding_key() -> str:
    """What the binding is compiled against: torch's C++ headers and the interpreter's."""
    import sysconfig

    import torch
    return "\n".join(str(x) for x in (torch.__version__, torch.__file__, torch._C._GLIBCXX_USE_CXX11_ABI,
                                      sysconfig.get_config_var("SOABI"), sysconfig.get_paths()["include"])) + "\n"


def _build_binding(force: bool) -> None:
    src = os.path.join(CSRC, "moe_binding.cpp")
    key = _binding_key()
    built = open(BINDING_KEY).read() if os.path.exists(BINDING_KEY) else ""
    if not (force or built != key or _stale(BINDING, [src, os.path.join(INCLUDE, "fp8q.h"), os.path.abspath(__file__)])):
        return
    import sysconfig

    import torch
    base = os.path.join(os.path.dirname(torch.__file__))
    tmp = BINDING + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-DTORCH_EXTENSION_NAME=_moe_binding",
           "-I", INCLUDE, "-isystem", os.path.join(base, "include"),
           "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(CUDA, "include"), "-isystem", sysconfig.get_paths()["include"],
           src, "-o", tmp, "-L", os.path.join(base, "lib"), "-lc10", "-lc10_cuda", "-ltorch", "-ltorch_cpu",
           "-ltorch_cuda", "-ltorch_python", "-L", PKG, "-l:libfp8q.so", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode:
        raise RuntimeError(f"g++ failed on {src}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    with open(BINDING_KEY, "w") as f:
        f.write(key)


def build(force: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()
    if force:
        for o in glob.glob(os.path.join(BUILD, "*.o")):
            os.remove(o)
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(_compile, srcs))
    if force or _stale(LIB, objs):
        tmp = LIB + ".tmp"
        subprocess.run([NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-Xcompiler", "-fPIC",
                        *objs, "-o", tmp], check=True)
        os.replace(tmp, LIB)
    _build_binding(force)
    with open(os.path.join(BUILD, "ptxas.log"), "w") as log:
        for o in objs:
            p = o + ".ptxas.txt"
            if os.path.exists(p):
                log.write(open(p).read())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv))
