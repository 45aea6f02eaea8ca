"""Build libswiglu.so (hipcc, gfx950) in-tree, next to this file.

    python -m swiglu_gated_mlp_amd.build

Three translation units, compiled side by side, export the C ABI of
include/swiglu.h: csrc/swiglu_api.hip (the products, kernels in
csrc/fused_kernels.hpp and csrc/product_kernels.hpp, adapters in
csrc/lora_*.hpp), csrc/train_api.hip (training, kernels in
csrc/train_kernels.hpp) and csrc/int8_api.hip (the int8 products, kernels in
csrc/int8_*.hpp and csrc/fused_kernels.hpp).
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_NAME = "libswiglu.so"
LIB_PATH = os.path.join(PKG, LIB_NAME)
SOURCES = [os.path.join(CSRC, f) for f in ("swiglu_api.hip", "train_api.hip", "int8_api.hip")]
ARCH = os.environ.get("SWIGLU_OFFLOAD_ARCH", "gfx950")


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found; ROCm is required to build libswiglu")


def compile_flags():
    return [
        "--offload-arch=%s" % ARCH, "-O3", "-std=c++17", "-fPIC",
        # no packed-fp32 instructions in device code
        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
        "-Wall", "-Wno-unused-result", "-I", INCLUDE, "-I", CSRC,
    ]


def link_flags():
    # the HIP runtime only: every kernel, the MLP block's down projection
    # included, is this library's own
    return []


def _run(cmd, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    out = "\n".join(l for l in res.stdout.splitlines()
                    if "packed-fp32-ops' is not a recognized feature" not in l)
    if res.returncode != 0:
        raise RuntimeError("hipcc failed (%d):\n%s" % (res.returncode, out))
    if verbose and out.strip():
        print(out, flush=True)


def build(verbose: bool = False) -> str:
    """Compile the library (always recompiles) and return its path."""
    tmp = LIB_PATH + ".tmp%d" % os.getpid()
    with tempfile.TemporaryDirectory(prefix="swiglu_build") as d:
        objs = [os.path.join(d, os.path.basename(s) + ".o") for s in SOURCES]
        with ThreadPoolExecutor(len(SOURCES)) as pool:
            list(pool.map(lambda so: _run([hipcc(), *compile_flags(), "-c", so[0], "-o", so[1]], verbose),
                          zip(SOURCES, objs)))
        _run([hipcc(), "--offload-arch=%s" % ARCH, "-shared", "-fPIC", "-o", tmp, *objs, *link_flags()], verbose)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
