"""Builds libecho.so (HIP, gfx950) in-tree with hipcc.

Every .hip file is compiled for gfx950 with packed-FP32 instructions disabled; host-only .cpp
files are compiled with hipcc as plain C++; the objects are linked into
dsa_indexer_top_amd/libecho.so.  Objects go to _build/ at the repository root.  The native module
of the tensor calls (native/tensor_calls.cpp) becomes dsa_indexer_top_amd/_tensor_calls.so.
"""

import concurrent.futures as cf
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OUT = os.path.join(PKG, "libecho.so")
CALLS = os.path.join(PKG, "_tensor_calls.so")
BUILD = os.path.join(ROOT, "_build")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

COMMON = ["-O3", "-fPIC", "-std=c++17", "-Wall", "-Wno-unused-function",
          "-I" + os.path.join(ROOT, "include")]
# The block-scaled product adds every MFMA's result to vector registers at once: left to itself the
# compiler sends the results of workgroups with few waves through accumulation registers, one move
# and a wait per value.
EXTRA = {"matmul_fp8.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"]}
DEVICE = ["--offload-arch=gfx950", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]


def sources():
    return sorted(f for f in os.listdir(CSRC) if f.endswith((".hip", ".cpp")))


def _compile(src):
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC] + COMMON
    if src.endswith(".hip"):
        cmd += DEVICE + EXTRA.get(src, [])
    cmd += ["-c", os.path.join(CSRC, src), "-o", obj]
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError("hipcc failed for %s:\n%s\n%s" % (src, " ".join(cmd), p.stderr))
    return obj


def _tensor_calls():
    """The native module of the tensor calls: host C++ against torch's headers, no HIP."""
    import sysconfig
    import torch
    from torch.utils.cpp_extension import include_paths
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = CALLS + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-fPIC", "-shared", "-std=c++17", "-Wall", "-fvisibility=hidden",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI,
           *("-isystem" + p for p in include_paths()), "-I" + sysconfig.get_paths()["include"],
           os.path.join(PKG, "native", "tensor_calls.cpp"), "-o", tmp, "-L" + lib, "-ltorch_python", "-ltorch_cpu", "-lc10"]
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError("g++ failed for native/tensor_calls.cpp:\n%s\n%s" % (" ".join(cmd), p.stderr))
    os.replace(tmp, CALLS)
    return CALLS


def build(verbose=False):
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        calls = ex.submit(_tensor_calls)
        objs = list(ex.map(_compile, srcs))
    tmp = OUT + ".tmp"
    cmd = [HIPCC, "-shared", "-fPIC", "--offload-arch=gfx950", "-o", tmp] + objs
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (" ".join(cmd), p.stderr))
    os.replace(tmp, OUT)
    calls.result()                           # its failure leaves the library, which needs neither it nor torch
    if verbose:
        print("built", OUT, CALLS)
    return OUT


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
