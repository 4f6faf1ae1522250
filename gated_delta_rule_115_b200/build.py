"""Build libmuir.so in-tree with nvcc for sm_100a, and the native half of the Python binding
(``_attn.so``) with g++ against the installed torch.

Usage: ``python -m gated_delta_rule_115_b200.build [--force] [--debug]``.
The shared library lands next to this file; object files go to ``_build/``.
``--debug`` (with ``--force`` to rebuild every object) defines MUIR_DEBUG: the
C-ABI entry points then also ask the CUDA runtime where every pointer lives and
refuse, with MUIR_ERR_INVALID_ARG, memory the device cannot address.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OBJ = os.path.join(ROOT, "_build", "obj")
LIB = os.path.join(HERE, "libmuir.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-Xptxas", "-warn-spills"]


def _deps():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
                  + [os.path.join(ROOT, "include", "muir.h")])


def _compile(src: str, obj: str, extra):
    cmd = [NVCC] + ARCH + FLAGS + list(extra) + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return r.stderr


BINDING = os.path.join(HERE, "_attn.so")


def build_binding(force: bool = False) -> str:
    """``csrc/torch_binding.cpp`` -> ``_attn.so``; rebuilt when its sources change or when it
    was built for another torch."""
    import sysconfig
    import torch
    from torch.utils import cpp_extension
    src = os.path.join(CSRC, "torch_binding.cpp")
    stamp = os.path.join(OBJ, "torch_binding.stamp")
    built_for = f"torch {torch.__version__} python {sysconfig.get_python_version()}"
    newest = max(os.path.getmtime(p) for p in (src, os.path.join(ROOT, "include", "muir.h")))
    if (not force and os.path.exists(BINDING) and os.path.getmtime(BINDING) >= newest
            and os.path.exists(stamp) and open(stamp).read() == built_for):
        return BINDING
    os.makedirs(OBJ, exist_ok=True)
    tmp = BINDING + f".tmp{os.getpid()}"
    cuda_include = os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}"]
    for d in cpp_extension.include_paths() + [cuda_include, sysconfig.get_paths()["include"]]:
        cmd += ["-isystem", d]
    cmd += [src, "-o", tmp] + [f"-L{d}" for d in cpp_extension.library_paths()]
    cmd += ["-lc10", "-lc10_cuda", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {src}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    with open(stamp, "w") as f:
        f.write(built_for)
    return BINDING


def build(force: bool = False, debug: bool = False, verbose: bool = False) -> str:
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    os.makedirs(OBJ, exist_ok=True)
    extra = ["-DMUIR_DEBUG=1"] if debug else []
    dep_time = max(os.path.getmtime(p) for p in _deps())
    jobs = []
    objs = []
    for s in srcs:
        o = os.path.join(OBJ, os.path.basename(s)[:-3] + ".o")
        objs.append(o)
        if force or not os.path.exists(o) or os.path.getmtime(o) < max(os.path.getmtime(s), dep_time):
            jobs.append((s, o))
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=min(8, len(jobs))) as ex:
            for msg in ex.map(lambda j: _compile(j[0], j[1], extra), jobs):
                if verbose and msg:
                    print(msg, file=sys.stderr)
    if force or jobs or not os.path.exists(LIB) or os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [NVCC] + ARCH + ["-shared", "-o", tmp] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    build_binding(force)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, debug="--debug" in sys.argv, verbose=True)
    print(LIB)
