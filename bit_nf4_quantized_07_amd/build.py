"""Build libqlora.so (gfx950) from the HIP sources in csrc/ with hipcc, and
_calls.so, the C++ marshalling of the batched adapters' Python calls, with g++
and torch's headers.  The C library needs hipcc alone: it is built where the
other cannot be.

    python -m bit_nf4_quantized_07_amd.build [--verbose]

The library is written next to this file so that it travels with the source
tree.  Object files go to _build/ (not tracked).
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libqlora.so")
CALLS = os.path.join(HERE, "_calls.so")
SOURCES = ["quant_kernels.hip", "gemm_kernels.hip", "fwd_kernels.hip", "dx_kernels.hip", "adapter_kernels.hip", "gemv_kernels.hip", "elementwise.hip",
           "merge_kernels.hip", "dropout_kernels.hip", "batch_plan_kernels.hip", "batch_kernels.hip",
           "qlora_api.hip"]
ARCH = "gfx950"

COMMON = [
    "-O3", "-std=c++17", f"--offload-arch={ARCH}", "-fPIC",
    # correctly rounded fp32 division: the quantiser's n = w / absmax is
    # specified as IEEE division
    "-fhip-fp32-correctly-rounded-divide-sqrt",
    # no packed-fp32 VALU instructions in device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
]


def hipcc() -> str:
    for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("hipcc not found")


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [hipcc(), *COMMON, "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    # the host pass does not know the packed-fp32 feature and says so; drop that line
    err = "\n".join(l for l in r.stderr.splitlines() if "packed-fp32-ops" not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{err}")
    if verbose and err.strip():
        print(err, file=sys.stderr)
    return obj


def _build_calls(verbose: bool) -> bool:
    """csrc/calls.cpp against torch's and Python's headers (host code only; it
    gets the addresses of libqlora.so's functions when it is loaded).  Without
    torch there is nothing it could marshal."""
    try:
        import torch
    except ImportError as e:
        print(f"_calls.so left out, torch is missing: {e}", file=sys.stderr)
        return False
    root = os.path.dirname(torch.__file__)
    tmp = CALLS + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-fvisibility=hidden",
           "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           f"-I{root}/include", "-I/opt/rocm/include", f"-I{sysconfig.get_paths()['include']}",
           os.path.join(CSRC, "calls.cpp"), "-o", tmp, f"-L{root}/lib", "-ltorch_python",
           "-ltorch_cpu", "-lc10", "-lc10_hip"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on calls.cpp:\n{r.stderr}")
    os.replace(tmp, CALLS)
    return True


def build(verbose: bool = False) -> str:
    """Compile every source and link the shared libraries; returns libqlora.so's
    path.  Raises after libqlora.so is linked where only _calls.so failed."""
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        calls = ex.submit(_build_calls, verbose)
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    tmp = LIB + ".tmp"
    cmd = [hipcc(), "-shared", "-fPIC", f"--offload-arch={ARCH}", "-o", tmp, *objs]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    failed = calls.exception()
    if (failed is not None or not calls.result()) and os.path.exists(CALLS):
        os.remove(CALLS)   # an older one may call libqlora.so's functions otherwise
    if failed is not None:
        raise RuntimeError("libqlora.so is built, _calls.so (the batched adapters' Python calls) "
                           f"is not: {failed}") from failed
    return LIB


if __name__ == "__main__":
    print(build(verbose="--verbose" in sys.argv))
