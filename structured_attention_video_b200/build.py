"""Builds libmonarch.so in-tree with nvcc for sm_100a, and the torch binding next to it.

    python -m structured_attention_video_b200.build [--force]

Each .cu file under csrc/ compiles to an object in parallel; the objects link
into structured_attention_video_b200/_build/libmonarch.so (CUDA runtime linked
statically, so the library needs only the NVIDIA driver at run time).
csrc/torch_binding.cpp becomes a CPython module, monarch_torch.<python>.torch-<version>.so,
which marshals torch tensors onto the library's C ABI.  It is compiled against the installed
torch's headers, so each version of torch (and of Python) has a module of its own.  Where it
cannot be built (no torch, no headers), that is said and the library stands without it: the
C ABI and the Monarch attention need none, and the others fail to import.
"""
from __future__ import annotations

import concurrent.futures
import glob
import importlib.metadata
import os
import re
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
OUT_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(OUT_DIR, "libmonarch.so")


def _binding() -> str:
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        version = "none"
    return os.path.join(OUT_DIR, "monarch_torch.%s.torch-%s.so"
                        % (sys.implementation.cache_tag, re.sub(r"[^\w.]", "-", version)))


BINDING = _binding()
HEADERS = [os.path.join(os.path.dirname(PKG), "include", "monarch_attn.h")]

NVCC_FLAGS = ["-O3", "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo",
              "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(dep) > t for dep in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(OUT_DIR, exist_ok=True)
    srcs = sources()
    deps = srcs + glob.glob(os.path.join(CSRC, "*.cuh")) + HEADERS
    if not force and not _stale(LIB, deps):
        _try_binding(force)
        return LIB
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.basename(src).replace(".cu", ".o"))
        cmd = [nvcc, *NVCC_FLAGS, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s%s" % (src, res.stdout, res.stderr))
        return obj, res.stderr

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(srcs)) as ex:
        results = list(ex.map(compile_one, srcs))
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [nvcc, "-shared", "-gencode", "arch=compute_100a,code=sm_100a",
           *[o for o, _ in results], "-o", tmp]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("link failed:\n%s%s" % (res.stdout, res.stderr))
    os.replace(tmp, LIB)
    _try_binding(force)
    return LIB


def _try_binding(force: bool) -> None:
    try:
        _build_binding(force)
    except (ImportError, OSError, RuntimeError) as e:
        if os.path.exists(BINDING):   # older than its source
            os.remove(BINDING)
        sys.stderr.write("The torch binding was not built, so the window attention, the paged "
                         "attention and the rotary positions are not there: %s\n" % e)


def _build_binding(force: bool) -> None:
    src = os.path.join(CSRC, "torch_binding.cpp")
    if not force and not _stale(BINDING, [src] + HEADERS):
        return
    import sysconfig

    import torch

    root = os.path.dirname(torch.__file__)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    includes = [os.path.join(root, "include"), os.path.join(cuda, "include"),
                sysconfig.get_paths()["include"]]
    tmp = BINDING + ".tmp%d" % os.getpid()
    # (libmonarch.so is found next to the module; torch's libraries are loaded before it)
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           *[x for i in includes for x in ("-isystem", i)], src, "-o", tmp,
           "-L" + os.path.join(root, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu",
           "-ltorch_python", "-L" + OUT_DIR, "-l:libmonarch.so", "-Wl,-rpath,$ORIGIN"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("g++ failed for %s:\n%s%s" % (src, res.stdout, res.stderr))
    os.replace(tmp, BINDING)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
