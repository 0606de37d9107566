"""Build libconv_i8.so and libdense.so (HIP, gfx950 only) in-tree with hipcc."""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_DIR = os.path.join(PKG, "_lib")
LIB = os.path.join(LIB_DIR, "libconv_i8.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

SOURCES = [os.path.join(CSRC, "conv_i8.hip")]
HEADERS = [os.path.join(CSRC, f) for f in ("kernel_common.hpp", "igemm_kernel.hpp", "footprint_kernel.hpp", "pointwise_kernel.hpp", "mfma_ceiling_kernel.hpp", "direct_kernel.hpp", "wgrad_kernel.hpp", "tuned_tiles.inc",
                                               "repack_kernel.hpp")] + [
    os.path.join(INCLUDE, "conv_i8.h")]

# The dense layer and layer norm: a library of their own, one object per source
DENSE_CSRC = os.path.join(PKG, "csrc_dense")
DENSE_LIB = os.path.join(LIB_DIR, "libdense.so")
DENSE_SOURCES = [os.path.join(DENSE_CSRC, f) for f in ("linear.hip", "gemm_bf16.hip", "gemm_f16.hip", "gemm_i8.hip",
                                                      "norm.hip", "gemm_f8.hip", "fp8.hip", "residual_norm.hip", "residual_norm_bf16.hip", "residual_norm_f16.hip",
                                                      "residual_norm_f32.hip", "clip.hip")]
# ... and the Python module that hands tensors to it (host code only)
DENSE_BIND_SOURCE = os.path.join(DENSE_CSRC, "bind.cpp")
DENSE_BIND = os.path.join(LIB_DIR, "_dense.so")

HIP_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
    "-Wall", "-Wno-unused-function", "-Wno-inline-asm",
    # packed fp32 VALU forms are kept out of every device code object
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def _run(cmds: list, verbose: bool) -> None:
    """Runs the compiler commands side by side; raises if one fails."""
    started = []
    for cmd in cmds:
        if verbose:
            print(" ".join(cmd), flush=True)
        log = tempfile.TemporaryFile("w+")
        started.append((cmd, subprocess.Popen(cmd, stdout=log, stderr=subprocess.STDOUT), log))
    # the host pass does not know the packed-fp32 feature name; drop that noise
    noise = "is not a recognized feature for this target"
    failed = []
    for cmd, p, log in started:
        rc = p.wait()
        log.seek(0)
        msgs = [l for l in log.read().splitlines() if noise not in l]
        log.close()
        if rc != 0:
            failed += [f"{cmd[0]} ended with {rc}", *msgs]  # also one that was killed without a word
        elif verbose and msgs:
            print("\n".join(msgs))
    if failed:
        raise RuntimeError("the compiler failed:\n" + "\n".join(failed))


def bind_command(out: str) -> list:
    import torch

    base = os.path.dirname(torch.__file__)
    include = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
               "/opt/rocm/include", sysconfig.get_paths()["include"], INCLUDE]
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__=1",
            "-DUSE_ROCM=1", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *[f for i in include for f in ("-I", i)], DENSE_BIND_SOURCE, "-o", out, "-L", os.path.join(base, "lib"),
            "-ltorch_python", "-ltorch_hip", "-ltorch_cpu", "-ltorch", "-lc10", "-lc10_hip"]


def build(verbose: bool = False, dense_only: bool = False) -> str:
    """Compiles both libraries, all sources side by side (the convolution's
    takes minutes), or only the dense one."""
    os.makedirs(LIB_DIR, exist_ok=True)
    tmp, dense_tmp, bind_tmp = (f + ".tmp" for f in (LIB, DENSE_LIB, DENSE_BIND))
    if os.path.exists(tmp):
        os.remove(tmp)
    objects = [os.path.join(LIB_DIR, os.path.basename(s)[:-4] + ".o") for s in DENSE_SOURCES]
    compile_flags = [f for f in HIP_FLAGS if f != "-shared"]
    cmds = [] if dense_only else [[HIPCC, *HIP_FLAGS, "-I", INCLUDE, "-I", CSRC, *SOURCES, "-o", tmp]]
    cmds.append(bind_command(bind_tmp))
    cmds += [[HIPCC, *compile_flags, "-I", INCLUDE, "-I", DENSE_CSRC, "-c", s, "-o", o]
             for s, o in zip(DENSE_SOURCES, objects)]
    try:
        _run(cmds, verbose)
    finally:
        # the convolution's library does without the other one, and without a host compiler
        if not dense_only and os.path.exists(tmp):
            os.replace(tmp, LIB)
    _run([[HIPCC, "--offload-arch=gfx950", "-fPIC", "-shared", *objects, "-o", dense_tmp]], verbose)
    os.replace(dense_tmp, DENSE_LIB)
    os.replace(bind_tmp, DENSE_BIND)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, dense_only="--dense" in sys.argv))
