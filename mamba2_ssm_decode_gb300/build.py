"""Build the CUDA library libssu_gb300.so in-tree (sm_103a only).

Each translation unit under csrc/ is compiled by nvcc in parallel into
_build/, then linked into mamba2_ssm_decode_gb300/libssu_gb300.so.  No cmake,
no torch extension machinery: the library is plain C ABI (include/ssu.h).
The argument checks of the layer calls are a small CPython module beside it
(_layer_binding.so, csrc/layer_binding.cpp: g++ with torch's headers).

    python -m mamba2_ssm_decode_gb300.build [--force] [--ptxas-info]
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import os
import shutil
import importlib.util
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libssu_gb300.so")
HEADER = os.path.join(ROOT, "include", "ssu.h")
BINDING_SRC = os.path.join(CSRC, "layer_binding.cpp")
BINDING = os.path.join(PKG, "_layer_binding.so")
STAMP = os.path.join(BUILD, "layer_binding.torch")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-Xcompiler", "-Wall", "-Xcompiler", "-fvisibility=hidden"]
# export only the C ABI: hide the statically linked CUDA runtime's symbols
LINK_FLAGS = ["-Xlinker", "--exclude-libs,ALL"]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libssu_gb300.so")
    return path


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps():
    return [os.path.join(CSRC, f) for f in os.listdir(CSRC)
            if f.endswith((".cuh", ".h"))] + [HEADER, os.path.abspath(__file__)]


def _stale(target, inputs):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(i) > t for i in inputs)


def _compile(src, ptxas_info):
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
    if ptxas_info:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stderr


def _torch():
    """Where torch is installed, or None.  The library needs none: only the CPython
    module is built with torch's headers, and is left out without them."""
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec else None


def _torch_is(torch):
    """What the module's object file is good for: this torch, at this place."""
    with open(os.path.join(torch, "version.py")) as f:
        return f"{torch}\n{f.read()}"


def _compile_binding(torch):
    """csrc/layer_binding.cpp to an object file (linked once the library is there)."""
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    obj = os.path.join(BUILD, "layer_binding.o")
    include = [os.path.join(torch, "include"), os.path.join(cuda, "include"),
               sysconfig.get_paths()["include"]]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-Wall",
           *(f"-isystem{p}" for p in include), "-c", BINDING_SRC, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {BINDING_SRC}:\n{r.stdout}\n{r.stderr}")
    with open(STAMP, "w") as f:
        f.write(_torch_is(torch))
    return obj


def _binding_stale(torch, obj):
    if _stale(obj, [BINDING_SRC, HEADER, os.path.abspath(__file__)]) or not os.path.exists(STAMP):
        return True
    with open(STAMP) as f:
        return f.read() != _torch_is(torch)


def _link_binding(torch, obj):
    tmp = BINDING + f".{os.getpid()}.tmp"
    cmd = ["g++", "-shared", "-o", tmp, obj, f"-L{PKG}", "-l:libssu_gb300.so", "-Wl,-rpath,$ORIGIN",
           f"-L{os.path.join(torch, 'lib')}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of _layer_binding.so failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)


def build(force: bool = False, ptxas_info: bool = False, verbose: bool = False) -> str:
    """Compile (if anything changed) and return the path of libssu_gb300.so."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()
    deps = _deps()
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in srcs]
    todo = [s for s, o in zip(srcs, objs) if force or ptxas_info or _stale(o, [s, *deps])]
    torch = _torch()
    binding = os.path.join(BUILD, "layer_binding.o")
    bind = torch is not None and (force or _binding_stale(torch, binding))
    bound = None
    if todo or bind:
        jobs = len(todo) + bind
        with cf.ThreadPoolExecutor(max_workers=min(jobs, os.cpu_count() or 4)) as ex:
            bound = ex.submit(_compile_binding, torch) if bind else None
            for obj, log in ex.map(lambda s: _compile(s, ptxas_info), todo):
                if verbose or ptxas_info:
                    print(f"== {os.path.basename(obj)}\n{log}", file=sys.stderr)
    if force or todo or _stale(LIB, objs):
        tmp = LIB + f".{os.getpid()}.tmp"
        cmd = [nvcc(), *ARCH, "-shared", "-Xcompiler", "-fPIC", *LINK_FLAGS, "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    if torch is None:
        print("torch is not installed: built the C library alone", file=sys.stderr)
        return LIB
    if bound:
        bound.result()
    if force or _stale(BINDING, [binding, LIB]):
        _link_binding(torch, binding)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true")
    args = ap.parse_args()
    print(build(force=args.force, ptxas_info=args.ptxas_info, verbose=True))
