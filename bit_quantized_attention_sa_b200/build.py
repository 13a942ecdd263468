"""Build libsa.so (the C-ABI CUDA library) in-tree for sm_100a.

    python -m bit_quantized_attention_sa_b200.build [--force] [--verbose]

Each ``csrc/*.cu`` file is compiled separately with nvcc for ``sm_100a`` (no fast-math:
the prologue relies on IEEE division and round-to-nearest-even) and the objects are
linked into ``bit_quantized_attention_sa_b200/libsa.so`` with the CUDA runtime linked
statically, so the library loads next to any PyTorch build and from plain C.  The torch side
of the serving calls (``csrc/sa_torch.cpp``) becomes ``_sa_torch.so`` beside it, against the
installed PyTorch.
"""
from __future__ import annotations

import argparse
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libsa.so")
SOURCES = ["sa_api.cu", "sa_prologue.cu", "sa_attn.cu", "sa_mask.cu", "sa_w8a8.cu", "sa_sla.cu", "sa_peak.cu",
           "sa_rope.cu", "sa_cache.cu", "sa_cache_attn.cu", "sa_cache_chunk.cu"]
HEADERS = ["sa_ptx.cuh", "sa_internal.h", "sa_attn_pairs.cuh", "sa_attn_mpairs.cuh",
           "sa_cache_attn.cuh"]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=default",
    "-I", os.path.join(ROOT, "include"),
]


TORCH_EXT = os.path.join(PKG, "_sa_torch.so")
TORCH_EXT_FITS = os.path.join(BUILD, "_sa_torch.fits")  # what TORCH_EXT was built against


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _stale(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    hdrs = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(ROOT, "include", "sa.h")]
    objs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s] + hdrs + [__file__]):
            cmd = [nvcc()] + NVCC_FLAGS + (["-Xptxas", "-v"] if verbose else []) + ["-c", s, "-o", o]
            subprocess.run(cmd, check=True)
    if force or _stale(LIB, objs):
        cmd = [nvcc(), "-shared", "-gencode", "arch=compute_100a,code=sm_100a", "-cudart", "static", "-o", LIB + ".tmp"] + objs
        subprocess.run(cmd, check=True)
        os.replace(LIB + ".tmp", LIB)
    src = os.path.join(CSRC, "sa_torch.cpp")
    if force or _stale(TORCH_EXT, [src, os.path.join(ROOT, "include", "sa.h"), __file__]) or not _torch_ext_fits():
        build_torch_ext(src)
    return LIB


def _torch_ext_for() -> str:
    """What the torch side depends on beside its sources: the PyTorch and Python that would load it
    (looked up without importing PyTorch, unless nothing but PyTorch itself knows its version)."""
    from importlib import metadata, util

    where = util.find_spec("torch")
    try:
        version = metadata.version("torch")
    except metadata.PackageNotFoundError:
        import torch

        version = torch.__version__
    return f"torch {version} at {where.origin if where else None}, {sys.implementation.cache_tag}"


def _torch_ext_fits() -> bool:
    if not os.path.exists(TORCH_EXT_FITS):
        return False
    with open(TORCH_EXT_FITS) as f:
        return f.read() == _torch_ext_for()


def build_torch_ext(src: str) -> None:
    """The torch side of the serving calls, _sa_torch.so, against libsa.so beside it and the
    installed PyTorch (g++; no device code)."""
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths, library_paths

    cuda = os.path.dirname(os.path.dirname(nvcc())) if os.path.isabs(nvcc()) else "/usr/local/cuda"
    dirs = include_paths() + [sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-DTORCH_EXTENSION_NAME=_sa_torch",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    cmd += [x for d in dirs for x in ("-isystem", d)] + [src, "-o", TORCH_EXT + ".tmp"]
    cmd += [f"-L{d}" for d in library_paths()] + [f"-L{PKG}", "-l:libsa.so", "-lc10", "-lc10_cuda", "-ltorch_cpu",
                                                  "-ltorch", "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
    subprocess.run(cmd, check=True)
    os.replace(TORCH_EXT + ".tmp", TORCH_EXT)
    with open(TORCH_EXT_FITS, "w") as f:
        f.write(_torch_ext_for())


def main(argv=None) -> int:
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true", help="print ptxas register/smem usage")
    a = ap.parse_args(argv)
    print(build(force=a.force, verbose=a.verbose))
    return 0


if __name__ == "__main__":
    sys.exit(main())
