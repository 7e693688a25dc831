"""Ahead-of-time build of libsdm_gx_gemm.so, libsdm_delta.so and libsdm_block.so for gfx950 with hipcc (in-tree, no JIT cache)."""

from __future__ import annotations

import os
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

from . import _code_check

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_PATH = os.path.join(PKG, "libsdm_gx_gemm.so")
SOURCES = ("gx_gemm_kernel.hip", "gx_gemm_mfma.hip", "gx_gemm_api.cpp", "gx_pa2_kernel.hip", "gx_pa2_api.cpp")
# the gated delta rule and the block norm: a library of their own
DELTA_LIB_PATH = os.path.join(PKG, "libsdm_delta.so")
DELTA_SOURCES = ("gdr_chunk.hip", "gdr_scan.hip", "gdr_grad.hip", "gdr_step.hip", "gdr_api.cpp", "nrm_kernel.hip",
                 "nrm_api.cpp", "delta_host.cpp")
# the gated linear recurrence, rows in 8 bits and the gated feed-forward product: another
BLOCK_LIB_PATH = os.path.join(PKG, "libsdm_block.so")
BLOCK_SOURCES = ("ffn_product.hip", "glr_kernel.hip", "qnt_kernel.hip", "ffn_few.hip", "ffn_lay.hip", "glr_api.cpp",
                 "qnt_api.cpp", "ffn_api.cpp", "delta_host.cpp")
JOBS = 6    # compilers at once

# Numerics-relevant flags: no contraction or fast-math (the chain's fmaf and the final add are what runs), f32
# denormals kept, and no packed-FP32 instructions (scalar v_fma_f32 / v_fmac_f32 only).
HIP_FLAGS = (
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-ffp-contract=off",
    "-fno-fast-math",
    "-fno-gpu-flush-denormals-to-zero",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-fvisibility=hidden",
    "-Wall",
)


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (ROCm is required to build libsdm_gx_gemm)")


def llvm() -> str:
    return os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin")


def build(out: str = LIB_PATH, verbose: bool = False, sources=SOURCES, check=None) -> str:
    """Compile every source for gfx950 and link the shared library (always recompiles). check(path) may refuse the linked
    library by an exception: then what was at `out` stays."""
    tmpdir = os.path.join(PKG, "_objs")
    os.makedirs(tmpdir, exist_ok=True)
    cc = hipcc()

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)

    def one(src):
        obj = os.path.join(tmpdir, os.path.splitext(src)[0] + ".o")
        lang = ["-x", "hip"] if src.endswith(".hip") else []
        run([cc, *HIP_FLAGS, "-I", INCLUDE, *lang, "-c", os.path.join(CSRC, src), "-o", obj])
        return obj

    with ThreadPoolExecutor(JOBS) as pool:
        objs = list(pool.map(one, sources))
    tmp = out + ".tmp"
    run([cc, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs])
    try:
        if check is not None:
            check(tmp)
        os.replace(tmp, out)
    finally:
        if os.path.exists(tmp):
            os.remove(tmp)
    return out


def build_delta(out: str = DELTA_LIB_PATH, verbose: bool = False, sources=DELTA_SOURCES) -> str:
    """The same for the gated delta rule and the block norm, whose machine code is checked (_code_check.py)."""
    return build(out, verbose, sources, lambda path: _code_check.verify(path, llvm()))


def build_block(out: str = BLOCK_LIB_PATH, verbose: bool = False, sources=BLOCK_SOURCES) -> str:
    """The same for the gated linear recurrence, rows in 8 bits and the gated feed-forward product, with the same check."""
    return build(out, verbose, sources, lambda path: _code_check.verify(path, llvm(), _code_check.BLOCK_WAITS))


if __name__ == "__main__":
    print(build(verbose=True))
    print(build_delta(verbose=True))
    print(build_block(verbose=True))
