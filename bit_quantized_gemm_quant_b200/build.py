"""Build libbqgemm.so in-tree with nvcc for sm_100a (cross-compiles without a GPU), and the
CPython marshalling of its fused products (_binding.so) with g++ against PyTorch's headers."""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libbqgemm.so")
MAIN = os.path.join(CSRC, "bqgemm.cu")
BINDING = os.path.join(PKG, "_binding.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-shared", "--expt-relaxed-constexpr",
]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libbqgemm.so")


def _sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(INCLUDE, "*.h")))


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(s) <= t for s in _sources())


def _binding_key() -> str:
    """What the binding is compiled against: a change of PyTorch or Python needs a new one."""
    import torch
    return f"torch {torch.__version__} {sysconfig.get_config_var('SOABI')}"


def _build_binding(force: bool, verbose: bool) -> None:
    deps = [BINDING_SRC, *glob.glob(os.path.join(INCLUDE, "*.h"))]
    stamp = os.path.join(os.path.dirname(BINDING), "_build", "binding.txt")      # the key of the built one
    key, built = _binding_key(), ""
    if os.path.exists(stamp):
        with open(stamp) as f:
            built = f.read()
    if (not force and built == key and os.path.exists(BINDING)
            and all(os.path.getmtime(s) <= os.path.getmtime(BINDING) for s in deps)):
        return
    import torch
    torch_root = os.path.dirname(torch.__file__)
    cuda_root = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    incs = [os.path.join(torch_root, "include"), os.path.join(torch_root, "include", "torch", "csrc", "api", "include"),
            os.path.join(cuda_root, "include"), sysconfig.get_paths()["include"]]
    tmp = BINDING + ".tmp"
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[a for i in incs for a in ("-isystem", i)], "-I", INCLUDE, BINDING_SRC, "-o", tmp,
           "-L" + os.path.join(torch_root, "lib"), "-lc10", "-ltorch_cpu", "-ltorch_python",
           "-lc10_cuda", "-L" + PKG, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd))
    subprocess.check_call(cmd)
    os.replace(tmp, BINDING)
    os.makedirs(os.path.dirname(stamp), exist_ok=True)
    with open(stamp, "w") as f:
        f.write(key)


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    if not force and up_to_date():
        _build_binding(False, verbose)
        return LIB
    tmp = LIB + ".tmp"
    cmd = [_nvcc(), *NVCC_FLAGS, *(extra_flags or []), "-I", INCLUDE, "-I", CSRC, MAIN, "-o", tmp]
    if verbose:
        print(" ".join(cmd))
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)
    _build_binding(force, verbose)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force=True, verbose=True, extra_flags=sys.argv[1:]))
