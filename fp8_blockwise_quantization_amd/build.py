"""Build the gfx950 HIP library ``libfp8rl.so`` in-tree with hipcc, and beside it the compiled argument
marshalling of the operators between the linears (``_marshal``, host code only) with the C++ compiler.

Usage: ``python -m fp8_blockwise_quantization_amd.build`` (or call ``build()``). With
``--library-only`` (``build(marshal=False)``) the library alone, for who calls the C ABI or the
linears' binding: the Python and torch headers, which the marshalling needs, may then be absent.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
LIB_NAME = "libfp8rl.so"
LIB_PATH = os.path.join(PKG_DIR, LIB_NAME)
SOURCES = ("quant.hip", "tensor_quant.hip", "transpose_quant.hip", "gemm.hip", "fp8rl_abi.hip",
           "norm.hip", "moe.hip", "rope_append.hip", "block_abi.hip")
MARSHAL_SOURCE = os.path.join(CSRC, "marshal.cpp")
MARSHAL_PATH = os.path.join(PKG_DIR, "_marshal" + sysconfig.get_config_var("EXT_SUFFIX"))
ARCH = "gfx950"

# -packed-fp32-ops: keep the compiler from forming packed FP32 instructions.
HIPCC_FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    "-Wall",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def hipcc_path() -> str:
    for cand in (shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found: the HIP toolchain (ROCm) is required to build libfp8rl")


def cxx_path() -> str:
    """A host C++ compiler: the system's, else the one that comes with hipcc."""
    for name in ("g++", "c++", "clang++", "amdclang++"):
        if path := shutil.which(name):
            return path
    path = os.path.join(os.path.dirname(hipcc_path()), "amdclang++")
    if os.path.exists(path):
        return path
    raise RuntimeError("a C++ compiler is required to build the argument marshalling")


def _run(cmd, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed with status {res.returncode}")


def build_marshal(verbose: bool = False) -> str:
    """Compile csrc/marshal.cpp against the installed torch and the library next to this file;
    returns the extension module's path."""
    import torch

    troot = os.path.dirname(torch.__file__)
    tmp = MARSHAL_PATH + ".tmp"
    cmd = [cxx_path(), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", os.path.join(ROOT, "include"), "-isystem", os.path.join(troot, "include"),
           "-isystem", sysconfig.get_paths()["include"], MARSHAL_SOURCE, "-o", tmp,
           "-L", os.path.join(troot, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10",
           "-L", PKG_DIR, "-l:" + LIB_NAME, "-Wl,-rpath,$ORIGIN"]
    _run(cmd, verbose)
    os.replace(tmp, MARSHAL_PATH)
    return MARSHAL_PATH


def build(verbose: bool = False, extra_flags=(), out_path: str | None = None,
          marshal: bool = True) -> str:
    """Compile every HIP source into ``libfp8rl.so`` next to this file, and the marshalling module
    that links to it (unless ``marshal`` is false; with ``out_path``, the library alone into that
    file); returns the library's path."""
    srcs = [os.path.join(CSRC, s) for s in SOURCES]
    out = out_path or LIB_PATH
    tmp = out + ".tmp"
    cmd = [hipcc_path(), *HIPCC_FLAGS, *extra_flags, "-I", os.path.join(ROOT, "include"),
           "-o", tmp, *srcs]
    _run(cmd, verbose)
    os.replace(tmp, out)
    if out_path is None and marshal:
        build_marshal(verbose)
    return out


if __name__ == "__main__":
    if set(sys.argv[1:]) - {"--library-only"}:
        sys.exit("usage: python -m fp8_blockwise_quantization_amd.build [--library-only]")
    print(build(verbose=True, marshal="--library-only" not in sys.argv))
