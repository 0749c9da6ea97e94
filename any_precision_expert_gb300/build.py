"""Build the C-ABI library (libpw.so) in-tree with nvcc for sm_103a.

Each translation unit is compiled in parallel into ``_build/`` next to this
file and linked into ``libpw.so`` in the package directory (static CUDA
runtime, so the library only needs the driver at run time).  The marshalling
module ``_pw_torch.so`` (torch tensors to the C ABI) is compiled beside it.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libpw.so")
BINDING = os.path.join(PKG, "_pw_torch.so")

SOURCES = ["pw_runtime.cpp", "pw_pack.cpp", "pw_planner.cpp", "pw_kernels.cu", "pw_ffn.cu", "pw_decode.cu",
           "pw_prefill.cu", "pw_noalloc.cu", "pw_serve.cpp", "pw_rope.cu", "pw_attend.cu", "pw_attend_tc.cu", "pw_verify.cu",
           "pw_context.cpp", "pw_prompt.cu", "pw_logprob.cu", "pw_cache4.cu", "pw_evict.cu"]
# the planner compares doubles: no fused multiply-adds, so x86 and Arm hosts plan alike
SOURCE_FLAGS = {"pw_planner.cpp": ["-Xcompiler", "-ffp-contract=off"]}
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc():
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def _flags(extra=()):
    return ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC,
            "-DNDEBUG", *ARCH, *extra]


def _compile(src: str, extra, verbose: bool):
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [_nvcc(), *_flags([*extra, *SOURCE_FLAGS.get(src, [])]), "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stderr


def _torch_object(verbose: bool) -> str:
    """Compile the marshalling module's one source against torch's headers."""
    from torch.utils import cpp_extension as ext
    obj = os.path.join(BUILD, "pw_torch.o")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-DNDEBUG", "-I", INCLUDE,
           *[a for p in ext.include_paths() for a in ("-isystem", p)], "-isystem", cuda,
           "-isystem", sysconfig.get_paths()["include"], "-c", os.path.join(CSRC, "pw_torch.cpp"), "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for pw_torch.cpp:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_binding(obj: str, verbose: bool) -> None:
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + ".tmp"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", PKG, "-l:libpw.so", "-Wl,-rpath,$ORIGIN", "-L", libs, "-lc10",
           "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)


def build(verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile every source and link libpw.so; returns the library path."""
    os.makedirs(BUILD, exist_ok=True)
    extra = ["-Xptxas", "-v"] if ptxas_info else []
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(_torch_object, verbose)
        results = list(ex.map(lambda s: _compile(s, extra, verbose), SOURCES))
    if ptxas_info:
        for _, err in results:
            sys.stderr.write(err)
    tmp = LIB + ".tmp"
    cmd = [_nvcc(), "-shared", *ARCH, "--cudart", "static", "-Xlinker", "-soname=libpw.so", "-o", tmp] + [o for o, _ in results]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _link_binding(binding.result(), verbose)
    return LIB


if __name__ == "__main__":
    build(verbose=True, ptxas_info="-v" in sys.argv)
