"""Builds libvggt_attn.so in-tree with nvcc for sm_100a, and _streaming.so, the
torch side of the streaming calls, with g++.

    python -m feed_forward_view_vggt_b200.build [--verbose] [--debug]

--debug builds libvggt_attn_debug.so with -DVGGT_DEBUG (device index checks).

The CUDA runtime is linked statically and the driver's tensor-map encoder
is fetched at run time, so the library loads (for symbol checks) on a
machine without a GPU driver.
"""
from __future__ import annotations

import argparse
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libvggt_attn.so")
# -DVGGT_DEBUG: device index checks reporting through the error word
DEBUG_LIB = os.path.join(HERE, "libvggt_attn_debug.so")
SOURCES = [os.path.join(CSRC, "vggt_attn.cu")]
DEPS = SOURCES + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))] + \
    [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]

# torch-side marshalling of the streaming calls (a Python extension module)
BINDING = os.path.join(HERE, "_streaming.so")
BINDING_SOURCE = os.path.join(CSRC, "streaming_binding.cpp")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-shared", "-Xcompiler", "-fPIC,-fvisibility=hidden",
    "-cudart", "static",
    "--expt-relaxed-constexpr",
]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(p) <= t for p in DEPS)


def build(force: bool = False, verbose: bool = False, debug: bool = False) -> str:
    """Builds the release library, or with debug=True the library with
    device index checks (-DVGGT_DEBUG), then the torch-side module, which
    alone needs torch and a host compiler; returns the library's path."""
    lib = DEBUG_LIB if debug else LIB
    if force or not up_to_date(lib):
        build_library(lib, verbose, debug)
    build_binding(force=force and not debug, verbose=verbose)
    return lib


def build_library(lib: str, verbose: bool = False, debug: bool = False) -> None:
    tmp = lib + ".tmp.%d" % os.getpid()
    cmd = [nvcc(), *NVCC_FLAGS, *(["-DVGGT_DEBUG"] if debug else []), "-I", INCLUDE, "-I", CSRC, "-o", tmp,
           *SOURCES]
    if verbose:
        cmd[1:1] = ["-Xptxas", "-v"]
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, lib)


def binding_is_for() -> str:
    """What the torch-side module is built for; it holds these words."""
    import torch

    return "built for torch %s, abi %d, %s" % (torch.__version__, torch._C._GLIBCXX_USE_CXX11_ABI,
                                               sys.implementation.cache_tag)


def binding_up_to_date() -> bool:
    if not os.path.exists(BINDING):
        return False
    deps = [BINDING_SOURCE] + [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    if any(os.path.getmtime(BINDING) < os.path.getmtime(p) for p in deps):
        return False
    with open(BINDING, "rb") as f:
        return binding_is_for().encode() in f.read()


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """Builds the torch-side module of the streaming calls; returns its path."""
    if not force and binding_up_to_date():
        return BINDING
    import sysconfig

    import torch

    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc())) if os.path.isabs(nvcc()) else "/usr/local/cuda"
    tmp = BINDING + ".tmp.%d" % os.getpid()
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI,
           '-DVGGT_BUILT_FOR="%s"' % binding_is_for(),
           "-isystem", os.path.join(root, "include"),
           "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"), "-isystem", sysconfig.get_paths()["include"], "-I", INCLUDE,
           "-o", tmp, BINDING_SOURCE, "-L", os.path.join(root, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu",
           "-ltorch_cuda", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, BINDING)
    return BINDING


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--debug", action="store_true", help="build libvggt_attn_debug.so (-DVGGT_DEBUG)")
    a = ap.parse_args()
    print(build(force=a.force or a.verbose, verbose=a.verbose, debug=a.debug))
