"""Build libwq.so (the HIP library behind include/wq.h) in-tree for gfx950.

Usage: python -m weight_only_bit_dequant_amd.build  (or __graft_entry__.build()).
Each source is compiled to an object in parallel, then linked into
weight_only_bit_dequant_amd/libwq.so; beside it _block_call.so, the CPython
entry points of block.py, is built against torch's headers.
"""

import concurrent.futures
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libwq.so")
EXT = os.path.join(HERE, "_block_call.so")

SOURCES = ["wq_api.hip", "wq_plan.cpp", "wq_quant.hip", "wq_linear.hip", "wq_gemm_tiled.hip", "wq_gemm_mid.hip", "wq_mx.hip", "wq_mlp.hip", "wq_noalloc.hip",
           "wq_block_api.hip", "wq_block_plan.cpp", "wq_block_quant.hip", "wq_block_gemm.hip"]

HIPCC = os.environ.get("HIPCC", shutil.which("hipcc") or "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    # correctly rounded fp32 division and IEEE denormals: quantized codes must
    # be bit-identical to an IEEE reference
    "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-fno-gpu-flush-denormals-to-zero",
    # keep the compiler from forming packed-fp32 VALU ops
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
    "-I", INCLUDE,
    "-I", CSRC,
]


def _compile(src):
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("hipcc failed for %s:\n%s\n%s" % (src, " ".join(cmd), r.stderr[-8000:]))
    return obj


def _build_ext():
    """_block_call.so: host code only, against the headers and libraries of the torch that will load it."""
    import torch
    from torch.utils import cpp_extension

    tmp = EXT + ".tmp"
    rocm = cpp_extension.ROCM_HOME or "/opt/rocm"
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI, "-I", INCLUDE]
    for path in [*cpp_extension.include_paths(), os.path.join(rocm, "include"), sysconfig.get_paths()["include"]]:
        cmd += ["-isystem", path]
    cmd += [os.path.join(CSRC, "wq_block_py.cpp"), "-o", tmp, "-L", libs, "-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("building _block_call failed:\n%s\n%s" % (" ".join(cmd), r.stderr[-8000:]))
    os.replace(tmp, EXT)
    return EXT


def build(verbose=False):
    os.makedirs(BUILD, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        ext = ex.submit(_build_ext)
        objs = list(ex.map(_compile, SOURCES))
        ext = ext.result()
    tmp = LIB + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (" ".join(cmd), r.stderr[-8000:]))
    os.replace(tmp, LIB)
    if verbose:
        print("built", LIB)
        print("built", ext)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
