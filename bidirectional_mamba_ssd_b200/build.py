"""Build libssd_bidir.so in-tree with nvcc for sm_100a, and the Python binding's
C++ part.

Each .cu under csrc/ is compiled to an object in _build/ and the objects are
linked into bidirectional_mamba_ssd_b200/libssd_bidir.so. Sources are rebuilt
when they (or a header) are newer than their object. csrc/ssd_binding.cpp
(torch's C++ headers, no CUDA code) becomes the extension module _binding beside
it; it is rebuilt as well when torch or Python are other ones than it was built for.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import re
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libssd_bidir.so")
BINDING = os.path.join(PKG, "_binding" + sysconfig.get_config_var("EXT_SUFFIX"))
BINDING_KEY = os.path.join(PKG, "_binding.key")     # what BINDING was built for
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def _newest_header() -> float:
    hs = glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))
    return max((os.path.getmtime(h) for h in hs), default=0.0)


def build(verbose: bool = False, extra_flags=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    hdr_t = _newest_header()
    objs = []
    for src in srcs:
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        objs.append(obj)
        if os.path.exists(obj) and os.path.getmtime(obj) >= max(os.path.getmtime(src), hdr_t) \
                and not extra_flags:
            continue
        cmd = [NVCC, *FLAGS, *extra_flags, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        subprocess.run(cmd, check=True)
    if (not os.path.exists(LIB) or any(os.path.getmtime(o) > os.path.getmtime(LIB) for o in objs)
            or extra_flags):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [NVCC, *ARCH, "-shared", "-o", tmp, *objs]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        subprocess.run(cmd, check=True)
        os.replace(tmp, LIB)
    build_binding(verbose)
    return LIB


def _torch_dir() -> str:
    return importlib.util.find_spec("torch").submodule_search_locations[0]


def _torch_version() -> str:
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        return re.search(r"__version__\s*=\s*['\"]([^'\"]+)", f.read()).group(1)


def build_binding(verbose: bool = False) -> str:
    src = os.path.join(CSRC, "ssd_binding.cpp")
    version = _torch_version()
    key = f"torch {version}, Python {sys.version}\n"
    built = None
    if os.path.exists(BINDING) and os.path.exists(BINDING_KEY):
        with open(BINDING_KEY) as f:
            built = f.read()
    if built == key and os.path.getmtime(BINDING) >= max(os.path.getmtime(src), _newest_header()):
        return BINDING
    torch = _torch_dir()
    cuda = os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include")
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", f'-DSSD_TORCH_VERSION="{version}"', "-I", INCLUDE]
    for d in (sysconfig.get_paths()["include"], os.path.join(torch, "include"),
              os.path.join(torch, "include", "torch", "csrc", "api", "include"), cuda):
        cmd += ["-isystem", d]
    cmd += [src, "-o", tmp, "-L", os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, BINDING)
    with open(BINDING_KEY, "w") as f:
        f.write(key)
    untagged = os.path.join(PKG, "_binding.so")      # would be taken by a Python that BINDING is not for
    if os.path.exists(untagged):
        os.remove(untagged)
    return BINDING


if __name__ == "__main__":
    print(build(verbose=True, extra_flags=tuple(sys.argv[1:])))
