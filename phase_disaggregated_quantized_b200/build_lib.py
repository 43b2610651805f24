"""Build libnvq.so (the C-ABI library) in-tree with nvcc for sm_100a, and the
package's binding of its shortest calls (_binding.so) with the host compiler.

Usage: python -m phase_disaggregated_quantized_b200.build_lib
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig

from . import binding_fits, binding_tag

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, "libnvq.so")
BINDING = os.path.join(PKG, "_binding.so")
BINDING_SOURCE = os.path.join(PKG, "csrc", "binding.cpp")
SOURCES = [os.path.join(PKG, "csrc", f) for f in sorted(os.listdir(os.path.join(PKG, "csrc"))) if f.endswith((".cu", ".cuh"))]
NVCC_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-std=c++17", "-lineinfo",
              "-Xcompiler", "-fPIC", "-shared"]


def needs_build() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = SOURCES + [os.path.join(ROOT, "include", "nvq.h")]
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    if force or needs_build():
        nvcc = os.environ.get("NVCC", "nvcc")
        cmd = [nvcc, *NVCC_FLAGS, "-o", LIB + ".tmp", os.path.join(PKG, "csrc", "nvq_api.cu")]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        subprocess.run(cmd, check=True)
        os.replace(LIB + ".tmp", LIB)
    build_binding(force)
    return LIB


def build_binding(force: bool = False) -> str:
    header = os.path.join(ROOT, "include", "nvq.h")
    if not force and os.path.exists(BINDING) and binding_fits(BINDING) \
            and os.path.getmtime(BINDING) >= max(map(os.path.getmtime, (BINDING_SOURCE, header))):
        return BINDING
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    lib = os.path.join(root, "lib")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DNVQ_BINDING_TAG="{binding_tag()}"',
           *(f"-isystem{d}" for d in inc), BINDING_SOURCE, "-o", BINDING + ".tmp", f"-L{lib}", f"-Wl,-rpath,{lib}", "-lc10",
           "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    subprocess.run(cmd, check=True)
    os.replace(BINDING + ".tmp", BINDING)
    return BINDING


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
