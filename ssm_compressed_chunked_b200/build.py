"""Build libattamba.so and libattamba_checked.so in-tree with nvcc for sm_100a, and the
_binding module (argument marshalling for the SSM block's operators) with g++.

    python -m ssm_compressed_chunked_b200.build [--verbose]

The library links the CUDA runtime statically and resolves the driver's
tensor-map encoder at run time, so it needs only libc and the NVIDIA driver.
libattamba_checked.so is the same source compiled with ATTAMBA_CHECKED: the
kernels test their index computations against the arrays they address and
report a failure in the status word (ATTAMBA_DEV_BOUNDS) instead of making the
access.  It is a debugging build, selected with ATTAMBA_LIBRARY=checked.
"""

import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libattamba.so")
LIB_CHECKED = os.path.join(HERE, "libattamba_checked.so")
BINDING = os.path.join(HERE, "_binding.so")
SOURCES = ["abi.cu", "chunk_index.cu", "kv_ssm_scan.cu", "chunk_attn.cu", "decode.cu", "handoff.cu", "proj_gemm.cu", "causal_conv.cu",
           "selective_scan.cu", "clear_rows.cu", "block_norm.cu", "device.cu"]
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
         "-Xcompiler", "-fPIC", "-shared", "-cudart", "static", "-I", INCLUDE, "-I", CSRC]


def _nvcc(out, extra, verbose):
    cmd = [NVCC] + FLAGS + extra + (["-Xptxas", "-v"] if verbose else []) + \
        [os.path.join(CSRC, s) for s in SOURCES] + ["-o", out + ".tmp"]
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True), out


def _gxx(out):
    """The CPython module: torch's headers and libraries, no CUDA code."""
    import torch
    root = os.path.dirname(torch.__file__)
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include"), sysconfig.get_paths()["include"], INCLUDE]
    # the system's compiler, whatever CXX says: the module shares torch's C++ runtime, and a compiler that links one
    # of its own into it would leave two in the process
    cxx = "/usr/bin/g++" if os.path.exists("/usr/bin/g++") else "g++"
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"] + [f"-I{d}" for d in inc] + \
        [os.path.join(CSRC, "binding.cpp"), "-o", out + ".tmp", "-L" + os.path.join(root, "lib"), "-lc10", "-lc10_cuda",
         "-ltorch_cpu", "-ltorch_python"]
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True), out


def build(verbose=False):
    jobs = [_nvcc(LIB, [], verbose), _nvcc(LIB_CHECKED, ["-DATTAMBA_CHECKED"], verbose), _gxx(BINDING)]
    for proc, out in jobs:
        so, se = proc.communicate()
        if proc.returncode != 0:
            sys.stderr.write(so + se)
            raise RuntimeError(f"the compiler failed for {os.path.basename(out)}")
        os.replace(out + ".tmp", out)
        if verbose:
            sys.stderr.write(se)
    return LIB


if __name__ == "__main__":
    print(build(verbose="--verbose" in sys.argv))
