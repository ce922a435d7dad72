"""Build the sm_100a CUDA library ``libkroquant.so`` in-tree (beside this file), and the
binding's native part ``kq_binding.<torch version>.so``.

    python -m w4a4_mxfp4_post_b200.build [--force]

The library is a plain shared object with the C ABI of ``include/kroquant.h``;
it is compiled with nvcc for sm_100a only and links the CUDA runtime
statically, so loading it needs no torch and no GPU.  The native part of the
binding is host code against torch's headers and is built after the library.
Where torch is not installed it is left out; where it does not compile (a torch
without CUDA, no g++, no Python headers) it is left out with a warning.  The
Python binding then does its calls.
"""
from __future__ import annotations

import os
import subprocess
import sys
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
INCLUDE = os.path.join(ROOT, "include")
SOURCES = [os.path.join(HERE, "csrc", "kroquant.cu")]
HEADERS = [os.path.join(INCLUDE, "kroquant.h")] + sorted(
    os.path.join(HERE, "csrc", f) for f in os.listdir(os.path.join(HERE, "csrc")) if f.endswith((".cuh", ".h")))
LIB = os.path.join(HERE, "libkroquant.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    "-Xptxas", "-warn-spills",
    "-cudart", "static",
]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(p) > t for p in SOURCES + HEADERS + [os.path.abspath(__file__)])


def binding_path() -> str:
    """The binding's native part: torch's ABI is in the name, for a file built against another must not load."""
    from importlib.metadata import version

    return os.path.join(HERE, f"kq_binding.{version('torch')}.so")


def build_binding(force: bool = False) -> str | None:
    """Compile csrc/binding.cpp; None without torch."""
    import importlib.util
    import sysconfig

    spec = importlib.util.find_spec("torch")
    if spec is None:
        return None
    out, src = binding_path(), os.path.join(HERE, "csrc", "binding.cpp")
    deps = [src, os.path.join(INCLUDE, "kroquant.h"), os.path.abspath(__file__)]
    if not force and os.path.exists(out) and all(os.path.getmtime(p) <= os.path.getmtime(out) for p in deps):
        return out
    if os.path.exists(out):
        os.remove(out)                       # if this build fails, nothing older is loaded in its place
    torch_dir = os.path.dirname(spec.origin)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    tmp = out + ".tmp%d" % os.getpid()
    subprocess.run(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-I", INCLUDE, "-I", os.path.join(torch_dir, "include"),
                    "-I", os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
                    "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"), src,
                    "-L", os.path.join(torch_dir, "lib"), "-ltorch", "-ltorch_cpu", "-ltorch_python", "-lc10", "-lc10_cuda",
                    "-o", tmp], check=True)
    os.replace(tmp, out)
    return out


def build(force: bool = False, verbose: bool = False) -> str:
    if force or _stale():
        tmp = LIB + ".tmp%d" % os.getpid()
        cmd = [nvcc(), *NVCC_FLAGS, "-I", INCLUDE, *SOURCES, "-o", tmp]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        subprocess.run(cmd, check=True)
        os.replace(tmp, LIB)
    try:
        build_binding(force)
    except (subprocess.CalledProcessError, OSError, ImportError) as e:
        warnings.warn(f"the binding's native part is left out, it could not be built: {e}")
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
