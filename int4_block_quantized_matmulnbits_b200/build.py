"""Build libmnb.so (the CUDA kernels + C ABI) in-tree for sm_100a with nvcc.

    python -m int4_block_quantized_matmulnbits_b200.build [-v] [--debug]

--debug links libmnb_debug.so instead: the same library with device-side
index checks in the kernels listed in DEBUG_SOURCES.

Each .cu file compiles to an object under _build/, then one shared library is
linked next to this file.  CUDA runtime is linked statically, so the library
only needs the NVIDIA driver at run time.

The _binding module, linked next to it with g++, makes the paged cache's calls for
Python (csrc/binding.cpp).  It needs the Python and the torch that it was built
for, so its name carries the one (_binding.<tag>.so) and it checks the other; the
rest of the library needs neither.
"""
from __future__ import annotations

import importlib.util
import os
import re
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "libmnb.so")
BUILD = os.path.join(ROOT, "_build")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-Xptxas", "-warn-spills", "-I", os.path.join(ROOT, "include")]
SOURCES = ["api.cu", "quantize.cu", "gemv.cu", "gemv_tc.cu", "gemv_resident.cu", "gemv_chain.cu", "gemm_tcgen05.cu", "embed.cu", "gptq.cu",
           "paged.cu", "paged_attention.cu"]
HEADERS = ["common.cuh", "internal.h", "raise_limit.h"]


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


# The debug build (libmnb_debug.so) compiles these files with device-side index
# checks (MNB_DEVICE_CHECKS); every other object is the release one.
DEBUG_SOURCES = ["gemv_resident.cu"]
DEBUG_OUT = os.path.join(HERE, "libmnb_debug.so")


BINDING = os.path.join(HERE, "_binding" + sysconfig.get_config_var("EXT_SUFFIX"))


def torch_version(root):
    """__version__ of the torch in the folder `root`, without importing it."""
    with open(os.path.join(root, "version.py")) as f:
        return re.search(r"^__version__[^=]*= *['\"]([^'\"]+)['\"]", f.read(), re.M).group(1)


def build_binding(verbose: bool = False) -> str:
    """The _binding module (csrc/binding.cpp): the paged cache's calls for Python, against torch's headers and libmnb.so."""
    src, torch = os.path.join(CSRC, "binding.cpp"), os.path.dirname(importlib.util.find_spec("torch").origin)
    version = torch_version(torch)
    stamp = os.path.join(BUILD, "binding.torch")   # the torch that it was built for
    same = os.path.exists(stamp) and open(stamp).read() == version
    if not same or _stale(BINDING, [src, os.path.join(ROOT, "include", "mnb.h")]):
        inc, lib = os.path.join(torch, "include"), os.path.join(torch, "lib")
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall", "-Wextra",
               f'-DMNB_TORCH="{version}"', "-I", os.path.join(ROOT, "include"), "-isystem", sysconfig.get_paths()["include"],
               "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
               "-isystem", os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include"), src, "-o", BINDING + ".tmp",
               "-L", HERE, "-l:libmnb.so", "-Wl,-rpath,$ORIGIN", "-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cpu",
               "-ltorch_python"]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.check_call(cmd)
        os.replace(BINDING + ".tmp", BINDING)
        with open(stamp, "w") as f:
            f.write(version)
        old = os.path.join(HERE, "_binding.so")   # a name that any Python would load
        if os.path.exists(old):
            os.remove(old)
    return BINDING


def build(verbose: bool = False, ptxas_verbose: bool = False, debug: bool = False, binding: bool = True) -> str:
    os.makedirs(BUILD, exist_ok=True)
    hdrs = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(ROOT, "include", f) for f in ("mnb.h", "mnb_tune.h")]
    objs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        dbg = debug and src in DEBUG_SOURCES
        o = os.path.join(BUILD, src.replace(".cu", "_debug.o" if dbg else ".o"))
        objs.append(o)
        if _stale(o, [s] + hdrs) or ptxas_verbose:
            cmd = [NVCC, *ARCH, *FLAGS, *(["-DMNB_DEVICE_CHECKS=1"] if dbg else []), "-c", s, "-o", o]
            if ptxas_verbose:
                cmd += ["-Xptxas", "-v"]
            if verbose:
                print(" ".join(cmd), flush=True)
            subprocess.check_call(cmd)
    out = DEBUG_OUT if debug else OUT
    if _stale(out, objs):
        tmp = out + ".tmp"
        cmd = [NVCC, *ARCH, "-shared", "-o", tmp, *objs]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.check_call(cmd)
        os.replace(tmp, out)
    if binding and not debug:
        build_binding(verbose)
    return out


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, ptxas_verbose="--ptxas" in sys.argv, debug="--debug" in sys.argv))
