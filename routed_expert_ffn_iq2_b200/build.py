"""Build libredlite_moe.so in-tree with nvcc for sm_100a, and beside it the
Python marshaller of the token mixers (_marshal.so, host C++)."""

from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libredlite_moe.so")
MARSHAL = os.path.join(PKG, "_marshal.so")

CXX = os.environ.get("CXX", "g++")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
    "-I", os.path.join(ROOT, "include"),
]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + [os.path.join(ROOT, "include", "redlite_moe.h")]


def _newer(target: str, deps) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(p) <= os.path.getmtime(target) for p in deps)


def up_to_date() -> bool:
    return _newer(LIB, _deps())


def marshal_abi() -> str:
    """The Python and torch that _marshal.so has to be built against: its file name does not tell."""
    import torch

    return " ".join([sysconfig.get_config_var("EXT_SUFFIX"), torch.__version__,
                     f"cxx11abi={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"])


def marshal_abi_matches() -> bool:
    """Whether _marshal.so was built against this Python and torch (the binary holds what it was built against)."""
    try:
        with open(MARSHAL, "rb") as f:
            return f"redlite_marshal_abi:{marshal_abi()};".encode() in f.read()
    except OSError:
        return False


def build_marshal(force: bool = False) -> str:
    """_marshal.so against torch's headers and libredlite_moe.so (found beside it)."""
    src = os.path.join(CSRC, "marshal.cpp")
    if (not force and _newer(MARSHAL, [src, os.path.join(ROOT, "include", "redlite_moe.h")])
            and marshal_abi_matches()):
        return MARSHAL
    import torch

    if os.path.exists(MARSHAL):
        os.remove(MARSHAL)  # it is out of date, whether or not the build below goes through
    t = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(NVCC))
    inc = [os.path.join(ROOT, "include"), os.path.join(t, "include"),
           os.path.join(t, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include"),
           sysconfig.get_paths()["include"]]
    tmp = MARSHAL + ".tmp"
    r = subprocess.run([CXX, "-O2", "-std=c++17", "-fPIC", "-shared", *[a for i in inc for a in ("-isystem", i)],
                        f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DREDLITE_MARSHAL_ABI="{marshal_abi()}"', src, "-o", tmp,
                        "-L", PKG, "-l:libredlite_moe.so", "-Wl,-rpath,$ORIGIN", "-L", os.path.join(t, "lib"),
                        "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"],
                       stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if r.returncode != 0:
        raise RuntimeError("marshal.cpp failed:\n" + r.stdout.decode(errors="replace"))
    os.replace(tmp, MARSHAL)
    return MARSHAL


def _try_marshal(force: bool = False) -> None:
    """The library stands without the marshaller: what cannot be compiled against this torch costs the token mixers'
    Python calls alone (they raise), not the C ABI nor the routed layer."""
    try:
        build_marshal(force)
    except (ImportError, OSError, RuntimeError) as e:
        warnings.warn(f"the token mixers' Python calls are not available: {e}")


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        _try_marshal()
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    procs, objs = [], []
    for src in _sources():
        obj = os.path.join(OBJ, os.path.basename(src) + ".o")
        objs.append(obj)
        cmd = [NVCC, *FLAGS, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            failed.append((src, out.decode(errors="replace")))
        elif verbose and out:
            print(out.decode(errors="replace"), file=sys.stderr)
    if failed:
        raise RuntimeError("nvcc failed:\n" + "\n".join(f"{s}:\n{o}" for s, o in failed))
    tmp = LIB + ".tmp"
    subprocess.check_call([NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "--cudart", "static",
                           "-o", tmp, *objs])
    os.replace(tmp, LIB)
    _try_marshal(force)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
