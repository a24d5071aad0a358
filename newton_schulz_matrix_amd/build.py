"""Build libnsortho.so (HIP, gfx950) in-tree with hipcc, and the host module
that the package's block calls go through with g++ against this torch.

Usage: ``python -m newton_schulz_matrix_amd.build`` or ``build()``; for C
programs ``python newton_schulz_matrix_amd/build.py --library``, which needs
neither g++ nor torch.
"""

from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_NAME = "libnsortho.so"
LIB_PATH = os.path.join(PKG, LIB_NAME)
SOURCES = ["api.hip", "train.hip", "optim.hip", "resnorm.hip", "mlp.hip"] + [
    f"kern_{kind}_{t}.hip" for kind in ("mlp", "xent") for t in ("bf16", "f16", "f32")] + [f"kern_{kind}_{t}.hip" for kind in ("sym", "nt")
                         for t in ("f16_128", "f16_192", "f16_256", "f32_128", "f32_64")]

ARCH = "gfx950"

HIP_FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-mcode-object-version=5",
    # Packed fp32 arithmetic is left to the scalar forms.
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
]


MARSHAL_PATH = os.path.join(PKG, "_marshal.so")


def marshal_command() -> list:
    """Compiles the host module that checks the arguments of small calls
    against this Python and this torch."""
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths
    includes = [flag for path in include_paths() for flag in ("-isystem", path)]
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *includes,
            "-I", sysconfig.get_paths()["include"], os.path.join(CSRC, "marshal.cpp"), "-o", MARSHAL_PATH + ".tmp",
            "-L", os.path.join(torch.__path__[0], "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc",
                 shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (ROCm is required to build libnsortho)")


def _start(cmd: list, verbose: bool) -> subprocess.Popen:
    if verbose:
        print(" ".join(cmd), flush=True)
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)


def _finish(proc: subprocess.Popen, what: str, verbose: bool) -> None:
    text = proc.communicate()[0].decode(errors="replace")
    if proc.returncode != 0:
        raise RuntimeError(f"{what}:\n{text}")
    if verbose and text.strip():
        print(text, flush=True)


def build_library(verbose: bool = False, extra_flags=None) -> str:
    """Compile every HIP source and link libnsortho.so next to this file: all
    that a C program needs, with hipcc alone."""
    cc = hipcc()
    objs = [os.path.join(CSRC, os.path.splitext(src)[0] + ".o") for src in SOURCES]
    procs = [_start([cc, *HIP_FLAGS, *(extra_flags or []), "-I", INCLUDE, "-c", os.path.join(CSRC, src), "-o", obj], verbose)
             for src, obj in zip(SOURCES, objs)]
    for proc, src in zip(procs, SOURCES):
        _finish(proc, f"the compiler failed on {src}", verbose)
    tmp = LIB_PATH + ".tmp"
    _finish(_start([cc, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs], verbose), "link failed", verbose)
    os.replace(tmp, LIB_PATH)
    for obj in objs:
        os.remove(obj)
    return LIB_PATH


def build_marshal(verbose: bool = False) -> str:
    """Compile the host module next to this file; this takes g++ (or CXX),
    Python's headers and torch."""
    _finish(_start(marshal_command(), verbose), "the compiler failed on marshal.cpp", verbose)
    os.replace(MARSHAL_PATH + ".tmp", MARSHAL_PATH)
    return MARSHAL_PATH


def build(verbose: bool = False, extra_flags=None) -> str:
    """The library, then the host module, which is left out where there is no
    torch to load it.  Where it cannot be built this raises, with the library
    in place for C programs and for every call that does not go through it."""
    path = build_library(verbose, extra_flags)
    if importlib.util.find_spec("torch") is None:
        print("no torch: the host module of the package's block calls is left out", file=sys.stderr)
        return path
    try:
        build_marshal(verbose)
    except Exception as e:
        raise RuntimeError(f"{path} is built, but the host module of the package's block calls is not: {e}") from e
    return path


if __name__ == "__main__":
    print((build_library if "--library" in sys.argv else build)(verbose="-v" in sys.argv))
