"""Build ``libpkv.so`` in-tree with nvcc for sm_100a (B200), and ``_marshal``, the argument
marshalling of four of the Python binding's calls, with the host compiler (an extension
module of the interpreter that builds it, under its suffix).

    python -m paged_kv_cache_459_b200.build [--force] [--verbose-ptxas]

The library is a plain shared object with a C ABI (``include/pkv.h``); the
CUDA runtime is linked statically so it loads into any process (a PyTorch
process included) without a matching libcudart.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libpkv.so")
MARSHAL_SRC = os.path.join(CSRC, "marshal.c")
MARSHAL = os.path.join(HERE, "_marshal" + sysconfig.get_config_var("EXT_SUFFIX"))
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

NVCC_FLAGS = [
    "-O3", "-std=c++17", "-lineinfo",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-Xcompiler", "-fPIC,-fvisibility=hidden", "-shared", "-cudart", "static",
    "--expt-relaxed-constexpr",
    "-I", os.path.join(ROOT, "include"),
]


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    deps = sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
    deps.append(os.path.join(ROOT, "include", "pkv.h"))
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(d) > t for d in deps)


def build_marshal(force: bool = False) -> str:
    untagged = os.path.join(HERE, "_marshal.so")  # as once built: any interpreter would take it
    if os.path.exists(untagged):
        os.remove(untagged)
    deps = [MARSHAL_SRC, os.path.join(ROOT, "include", "pkv.h")]
    if not force and os.path.exists(MARSHAL) \
            and all(os.path.getmtime(d) <= os.path.getmtime(MARSHAL) for d in deps):
        return MARSHAL
    tmp = MARSHAL + f".tmp{os.getpid()}"
    subprocess.run(["gcc", "-O2", "-std=gnu11", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall", "-Wextra",
                    "-I", sysconfig.get_paths()["include"], "-o", tmp, MARSHAL_SRC], check=True)
    os.replace(tmp, MARSHAL)
    return MARSHAL


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    if force or _stale():
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [NVCC, *NVCC_FLAGS, *(["-Xptxas", "-v"] if verbose_ptxas else []), "-o", tmp, *sources()]
        subprocess.run(cmd, check=True)
        os.replace(tmp, LIB)
    build_marshal(force)  # after the library, which the other calls need alone
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="--verbose-ptxas" in sys.argv))
