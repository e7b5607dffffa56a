"""Build liblowbit.so (HIP, gfx950) in-tree with hipcc, and the Python
binding's compiled part (_marshal.so, host code against torch's headers)
with g++; where torch is absent the library alone.

Run ``python -m bit_matmul_lowbit_amd.build`` or call ``build()``.  Every call
recompiles.  Both are placed next to this file so that they travel with the
source tree.
"""
from __future__ import annotations

import importlib.util
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "liblowbit.so")
SOURCES = ["lowbit_api.cpp", "pack.hip", "gemv.hip", "gemv_mfma.hip", "gemv_small.hip", "gemm.hip", "ffn.hip", "ends.hip", "ternary.hip", "noalloc.hip", "norm.hip", "logits.hip", "lora.hip", "kv.hip", "attention.hip", "sample.hip", "probes.hip"]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    "-munsafe-fp-atomics",
    # packed FP32 instructions are kept out of the device code on purpose
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
]


MARSHAL = os.path.join(HERE, "_marshal.so")
CXX = os.environ.get("CXX", "g++")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")


def _run(cmd, out: str, verbose: bool) -> None:
    """Run a compiler that writes out + ".tmp", and move that to `out`."""
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"{cmd[0]} failed building {os.path.basename(out)}")
    os.replace(out + ".tmp", out)


def build_marshal(verbose: bool = False) -> str:
    import torch

    root = os.path.dirname(torch.__file__)
    inc, lib = os.path.join(root, "include"), os.path.join(root, "lib")
    # the torch libraries are found by their names, being loaded by then
    _run([CXX, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", inc,
          "-I", os.path.join(inc, "torch", "csrc", "api", "include"), "-I", sysconfig.get_paths()["include"],
          "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROCM, "include"), "-D__HIP_PLATFORM_AMD__",
          "-o", MARSHAL + ".tmp", os.path.join(CSRC, "marshal.cpp"), "-L", lib, "-ltorch_python", "-ltorch_cpu",
          "-lc10"], MARSHAL, verbose)
    return MARSHAL


def build(verbose: bool = False) -> str:
    """The library, which takes hipcc alone, and then, where there is a torch to
    call it from, the binding's compiled part."""
    srcs = [os.path.join(CSRC, s) for s in SOURCES]
    _run([HIPCC, *FLAGS, "-I", os.path.join(ROOT, "include"), "-o", LIB + ".tmp", *srcs], LIB, verbose)
    if importlib.util.find_spec("torch") is None:
        print("no torch here: _marshal.so, which the Python binding loads, is not built", file=sys.stderr)
    else:
        build_marshal(verbose)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
