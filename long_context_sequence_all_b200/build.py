"""Build ``libulysses.so`` (all CUDA sources, sm_100a) in-tree with nvcc.

    python -m long_context_sequence_all_b200.build [--force] [--verbose]

and ``_native.so``, the Python binding of the token-wise operators (g++).

Objects go to ``_build/``; the shared library lands next to this file so it
travels with the source tree.  nvcc cross-compiles for sm_100a without a GPU.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.metadata
import os
import re
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libulysses.so")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
NATIVE = os.path.join(HERE, "_native.so")         # Python binding of the token-wise operators
NATIVE_SRC = os.path.join(CSRC, "binding.cpp")

SOURCES = ["api.cu", "prof.cu", "permute.cu", "loss.cu", "loss_noalloc.cu", "attn_f32.cu", "attn_fwd_sm100.cu",
           "attn_bwd_sm100.cu", "attn_bwd_fused_sm100.cu", "proj_sm100.cu", "kv_copy.cu", "labels.cu",
           "tokenwise.cu", "norm.cu", "linear_sm100.cu", "linear_loss_sm100.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC",
         "-Xcompiler", "-Wall", "-I", INCLUDE]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _deps_mtime() -> float:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != os.path.basename(NATIVE_SRC)] + [os.path.join(INCLUDE, "ulysses.h")]
    return max(os.path.getmtime(f) for f in files)


# Kernels that split their register pool between warpgroups with setmaxnreg:
# the split only adds up when the kernel launches with exactly this many
# registers per thread; any other count would make setmaxnreg.inc wait forever.
REGISTER_SPLIT_KERNELS = {
    "attn_fwd_sm100.cu": [("attn_fwd_sm100_kernel", 168)],
    "attn_bwd_sm100.cu": [("attn_dkdv_sm100_kernel", 168), ("attn_dq_sm100_kernel", 168)],
    "attn_bwd_fused_sm100.cu": [("attn_bwd_sm100_kernel", 128)],
}


def _check_register_split(src: str, ptxas_log: str):
    lines = ptxas_log.splitlines()
    for kernel, want in REGISTER_SPLIT_KERNELS[src]:
        found = False
        # every instance of the kernel (template instantiations included)
        for i, line in enumerate(lines):
            if "Compiling entry function" in line and kernel in line:
                for nxt in lines[i + 1:i + 6]:
                    m = re.search(r"Used (\d+) registers", nxt)
                    if m:
                        if int(m.group(1)) != want:
                            raise RuntimeError(f"{kernel} uses {m.group(1)} registers, its warpgroup register "
                                               f"split needs exactly {want}; refusing to build")
                        found = True
                        break
        if not found:
            raise RuntimeError(f"ptxas report for {kernel} not found; refusing to build")


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, src.replace(".cu", ".o"))
    cmd = [nvcc(), *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose or src in REGISTER_SPLIT_KERNELS:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if src in REGISTER_SPLIT_KERNELS:
        _check_register_split(src, r.stdout + r.stderr)
    if verbose and (r.stdout or r.stderr):
        print(r.stdout + r.stderr, file=sys.stderr)
    return obj


def native_tag() -> str:
    """What a binding is built for, as it stands in ``_native.so``."""
    return f"ulysses binding: torch {importlib.metadata.version('torch')}, {sysconfig.get_config_var('SOABI')}"


def native_fits(path: str = None) -> bool:
    """Whether the built binding is for the torch and Python at hand."""
    with open(path or NATIVE, "rb") as f:
        return native_tag().encode() + b"\0" in f.read()


def build_native(force: bool = False) -> str:
    """The binding (g++ against the installed torch and Python)."""
    newest = max(os.path.getmtime(f) for f in (NATIVE_SRC, os.path.join(INCLUDE, "ulysses.h")))
    if not force and os.path.exists(NATIVE) and os.path.getmtime(NATIVE) >= newest and native_fits(NATIVE):
        return NATIVE
    import torch
    from torch.utils import cpp_extension
    inc = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(os.path.dirname(nvcc()), "..", "include"),
           *cpp_extension.include_paths()]
    lib = cpp_extension.library_paths()
    tmp = NATIVE + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DULY_BINDING_TAG="{native_tag()}"',
           *[x for d in inc for x in ("-isystem", d)], NATIVE_SRC, "-o", tmp,
           *[x for d in lib for x in (f"-L{d}", f"-Wl,-rpath,{d}")],
           "-lc10", "-lc10_cuda", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-ldl"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {NATIVE_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, NATIVE)
    return NATIVE


def build_library(force: bool = False, verbose: bool = False) -> str:
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= _deps_mtime():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-lcudart_static", "-ldl", "-lrt", "-lpthread"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


def build(force: bool = False, verbose: bool = False) -> str:
    """Both; the library, which needs nvcc alone, is there also where the binding fails."""
    path = build_library(force, verbose)
    build_native(force)
    return path


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
