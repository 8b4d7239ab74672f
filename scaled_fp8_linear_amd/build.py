"""Build ``libfp8lin.so`` (the gfx950 kernels and the C ABI) in-tree with hipcc, and
``_binding.so`` (the CPython side of the row operators) with g++ against torch's headers.

Usage: ``python -m scaled_fp8_linear_amd.build`` (or ``__graft_entry__.build()``).
Every call recompiles; object files go to ``scaled_fp8_linear_amd/_build/``. Without g++ or torch's
headers the library is still built, and the call ends with an error that says what is missing.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libfp8lin.so")
BINDING = os.path.join(PKG, "_binding.so")
ROOT = os.path.dirname(PKG)

SOURCES = ["abi.cpp", "quantize_amax.hip", "quantize_block.hip", "scale_update.hip",
           "pad_tokens.hip", "pad_varlen.hip", "gemm_fp8.hip", "bias.hip", "linear_small.hip",
           "layernorm.hip", "moe.hip"]

ARCH = "gfx950"
FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-fPIC", "-std=c++17",
    # hipcc fuses float32 code into packed-fp32 instructions on its own; keep them off.
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # scale arithmetic must use the correctly rounded float32 division
    "-fhip-fp32-correctly-rounded-divide-sqrt", "-fno-fast-math", "-ffp-contract=off",
    "-Wno-unused-command-line-argument",
    f"-I{os.path.join(ROOT, 'include')}",
]


def hipcc() -> str:
    for cand in (shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found: the ROCm toolchain is required to build libfp8lin.so")


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    lang = ["-x", "hip"] if src.endswith(".cpp") else []
    cmd = [hipcc()] + FLAGS + lang + ["-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def _compile_binding() -> None:
    import sysconfig

    import torch
    home = os.path.dirname(torch.__file__)
    lib = os.path.join(home, "lib")
    tmp = BINDING + ".tmp"
    cmd = ["g++", "-O2", "-fPIC", "-shared", "-std=c++17", "-fvisibility=hidden", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-isystem", os.path.join(home, "include"),
           "-isystem", sysconfig.get_paths()["include"],
           os.path.join(CSRC, "binding.cpp"), "-o", tmp, f"-L{lib}", f"-Wl,-rpath,{lib}",
           "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on binding.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(min(8, len(SOURCES) + 1)) as ex:
        binding = ex.submit(_compile_binding)
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    # the library does not need the binding, so it is there even if the binding cannot be built;
    # an older binding, which may not fit it, is not left beside it
    try:
        binding.result()
    except Exception as e:
        if os.path.exists(BINDING):
            os.remove(BINDING)
        raise RuntimeError(f"built {LIB}, but not {BINDING}, which the Python calls of the row "
                           f"operators need: {e}") from e
    if verbose:
        print(f"built {LIB}\nbuilt {BINDING}")
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
