"""Builds the C-ABI shared library libdm05_suffix_attn.so in-tree (sm_100a), which
needs nvcc alone, and where torch and Python's headers are installed the Python
module _torch_front, the torch front end of the prefix-cache operators (host
code)."""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libdm05_suffix_attn.so")
SOURCES = [os.path.join(HERE, "csrc", f) for f in ("dm05_suffix_attn.cu", "prefix_cache.cu")]


def deps() -> list:
    """Every file the library is compiled from: the sources, each header the
    sources include from csrc/, and the public header."""
    csrc = os.path.join(HERE, "csrc")
    inc = os.path.join(ROOT, "include")
    out = list(SOURCES)
    for d, exts in ((csrc, (".cuh", ".h")), (inc, (".h",))):
        out += [os.path.join(d, f) for f in sorted(os.listdir(d)) if f.endswith(exts)]
    return out


NVCC_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3", "-std=c++17",
              "-Xcompiler", "-fPIC", "-shared"]


FRONT_SOURCE = os.path.join(HERE, "csrc", "torch_front.cpp")


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def front_path() -> str:
    """Where the torch front end is built and loaded: it is C++ against this
    interpreter's and this torch's binary interface, whose versions its name
    carries, so that one built against others is never loaded."""
    import torch
    return os.path.join(HERE, f"_torch_front.{sysconfig.get_config_var('SOABI')}-torch-{torch.__version__}.so")


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile what is missing or older than a source file; the path of the library."""
    if force or not _fresh(LIB, deps()):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc(), *NVCC_FLAGS, "-I", os.path.join(ROOT, "include"), "-o", tmp, *SOURCES]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
            print(" ".join(cmd))
        subprocess.run(cmd, check=True)
        os.replace(tmp, LIB)
    why = front_unavailable()
    if why is None:
        build_front(force)
    else:
        print(f"the torch front end is not built: {why}", file=sys.stderr)
    return LIB


def _fresh(path: str, sources: list) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(d) <= os.path.getmtime(path) for d in sources)


def front_unavailable():
    """Why the torch front end cannot be built on this machine, or None."""
    try:
        import torch  # noqa: F401
    except ImportError:
        return "torch is not installed"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python.h is not installed"
    return None


def build_front(force: bool = False) -> str:
    """Compile the torch front end when it is missing or older than its sources;
    the path of this interpreter's and this torch's."""
    front = front_path()
    sources = [FRONT_SOURCE, os.path.join(ROOT, "include", "dm05_suffix_attn.h")]
    if not force and _fresh(front, sources):
        return front
    import torch
    home = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc())) or "/usr/local/cuda"
    include = [os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include"), os.path.join(ROOT, "include")]
    tmp = front + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           *[f"-I{d}" for d in include], FRONT_SOURCE, "-o", tmp, "-L" + os.path.join(home, "lib"), "-lc10",
           "-lc10_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python"]
    subprocess.run(cmd, check=True)
    os.replace(tmp, front)
    return front


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
