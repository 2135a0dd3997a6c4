"""Build librra.so (the CUDA library) in-tree for sm_103a with nvcc.

Every translation unit is compiled in parallel, then linked into one shared
library next to this file.  No CMake, no torch extension machinery: the
library has a plain C ABI (include/rra.h, include/rra_probe.h).
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "librra.so")
NATIVE = os.path.join(HERE, "_serve.so")  # the Python binding of rra_serve.h

SOURCES = ["kernels.cu", "cluster.cu", "coll.cu", "fused.cu", "rra_api.cu", "probes.cu", "rra_static.cu", "serve.cu",
           "serve_attn.cu", "serve_prefill.cu", "serve_attn_team.cu"]
HEADERS = ["prims.cuh", "cluster_prims.cuh", "rra_internal.h", "placement.h", "kernel_attrs.h", "serve_common.cuh",
           "serve_attn.cuh", "serve_attn_rows.cuh"]
PUBLIC_HEADERS = ["rra.h", "rra_probe.h", "rra_static.h", "rra_device.cuh", "rra_serve.h"]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--expt-relaxed-constexpr", "-I" + INCLUDE, "-I" + CSRC]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build librra.so")
    return path


def _newest_input() -> float:
    files = [os.path.join(CSRC, f) for f in SOURCES + HEADERS + ["serve_bind.cpp"]]
    files += [os.path.join(INCLUDE, f) for f in PUBLIC_HEADERS]
    files.append(os.path.abspath(__file__))
    return max(os.path.getmtime(f) for f in files)


def _native_command(out: str) -> list:
    """The compiler's command for _serve.so, against the installed torch (for its tensors' types and the current stream)."""
    import torch

    at = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    include = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(at, "include"),
               os.path.join(at, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include")]
    return ["g++", "-O2", "-std=c++17", "-Wall", "-shared", "-fPIC", "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI,
            *("-I" + i for i in include), os.path.join(CSRC, "serve_bind.cpp"), "-o", out, "-L" + os.path.join(at, "lib"),
            "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-ldl", "-Wl,-rpath," + os.path.join(at, "lib")]


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile and link; returns the path of librra.so.  Skips work when the
    library is newer than every source."""
    if not force and all(os.path.exists(f) and os.path.getmtime(f) >= _newest_input() for f in (LIB, NATIVE)):
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    procs = []
    objs = []
    for src in SOURCES:
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        objs.append(obj)
        cmd = [cc, *ARCH, *FLAGS, *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    native = NATIVE + ".tmp%d" % os.getpid()
    procs.append(("serve_bind.cpp", subprocess.Popen(_native_command(native), stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    errors = []
    for src, p in procs:
        out, _ = p.communicate()
        text = out.decode(errors="replace")
        if p.returncode != 0:
            errors.append("%s:\n%s" % (src, text))
        elif verbose and text.strip():
            print(text, file=sys.stderr)
    if errors:
        raise RuntimeError("nvcc failed\n" + "\n".join(errors))
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [cc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    p = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if p.returncode != 0:
        raise RuntimeError("link failed:\n" + p.stdout.decode(errors="replace"))
    os.replace(tmp, LIB)
    os.replace(native, NATIVE)
    return LIB


if __name__ == "__main__":
    force = "--force" in sys.argv
    print(build(force=force, verbose=True))
