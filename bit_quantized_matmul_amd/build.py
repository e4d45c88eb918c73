"""Build libbqm.so (the HIP kernels and the C ABI) for gfx950, in-tree.

Usage: ``python -m bit_quantized_matmul_amd.build`` (also called by
``__graft_entry__.build()``).  Every HIP source under ``csrc/`` is compiled with
hipcc for gfx950 only, then linked into ``bit_quantized_matmul_amd/libbqm.so``.  That
needs nothing else.  Then ``csrc/calls.cpp``, the binding's calls that are made for
every token, becomes ``bit_quantized_matmul_amd/_calls.so``, with g++ and PyTorch's
headers: without PyTorch it is left out, and a failure there leaves the library
in place.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libbqm.so")
CALLS = os.path.join(PKG, "_calls.so")
ARCH = "gfx950"

COMMON = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
    # correctly rounded fp32 division (the A8 and Q4_0 encoders rely on it)
    "-fhip-fp32-correctly-rounded-divide-sqrt",
    # no packed fp32 instructions anywhere (hipcc's host pass warns: harmless)
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", INCLUDE, "-I", CSRC,
]
# sources whose results must be bit-exact: no fused multiply-add contraction
EXACT = {"act_quant.hip", "cq_pack.hip", "codebook_fit.hip", "q4_0.hip"}


def hipcc() -> str:
    path = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(path):
        raise RuntimeError("hipcc not found: the HIP toolchain is required to build libbqm")
    return path


def sources() -> list[str]:
    """All HIP sources, the long compiles (GEMV kernel sets, GEMM) first."""
    srcs = sorted(f for f in os.listdir(CSRC) if f.endswith(".hip"))
    return sorted(srcs, key=lambda f: (not f.startswith("cq_gemv_i"), f != "cq_gemm.hip", f))


def _compile(src: str) -> str:
    obj = os.path.join(BUILD_DIR, src.replace(".hip", ".o"))
    flags = list(COMMON)
    if src in EXACT:
        flags.append("-ffp-contract=off")
    cmd = [hipcc(), *flags, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{r.stderr}")
    return obj


def _compile_calls() -> str | None:
    """The extension under a temporary name; None without PyTorch."""
    try:
        import torch
    except ImportError:
        return None
    from torch.utils.cpp_extension import include_paths, library_paths
    tmp = CALLS + ".tmp"
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-I{d}" for d in (INCLUDE, *include_paths(), sysconfig.get_paths()["include"])),
           os.path.join(CSRC, "calls.cpp"), "-o", tmp, *(f"-L{d}" for d in library_paths()),
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on calls.cpp:\n{r.stderr}")
    return tmp


def build(verbose: bool = True) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs = sources()
    jobs = min(len(srcs), max(1, min(8, os.cpu_count() or 1)))
    with ThreadPoolExecutor(max_workers=jobs) as ex:
        calls = ex.submit(_compile_calls)                        # beside the library's sources
        objs = list(ex.map(_compile, srcs))
    tmp = LIB + ".tmp"
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB} from {len(srcs)} sources", file=sys.stderr)
    if os.path.exists(CALLS):
        os.remove(CALLS)                                         # an earlier library's
    tmp = calls.result()
    if tmp:
        os.replace(tmp, CALLS)
    else:
        print("PyTorch is not installed: the binding's extension is left out", file=sys.stderr)
    return LIB


if __name__ == "__main__":
    build()
