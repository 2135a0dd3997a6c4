"""Build librra.so (the CUDA library) in-tree for sm_103a with nvcc.

Every translation unit is compiled in parallel, then linked into one shared
library next to this file.  No CMake, no torch: the library has a plain C ABI
(include/rra.h, include/rra_serve.h, include/rra_probe.h).  Where torch is
installed, _serve.so is compiled against it as well: the Python binding of
rra_serve.h, which reads tensors themselves.
"""
from __future__ import annotations

import importlib.util
import os
import re
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
NATIVE_STAMP = os.path.join(BUILD, "_serve.torch")  # the torch that it was built against

SOURCES = ["kernels.cu", "cluster.cu", "coll.cu", "fused.cu", "rra_api.cu", "probes.cu", "rra_static.cu", "serve.cu",
           "serve_attn.cu", "serve_prefill.cu", "serve_attn_team.cu", "serve_kv8.cu", "serve_pages.cu",
           "serve_prompt.cu"]
HEADERS = ["prims.cuh", "cluster_prims.cuh", "rra_internal.h", "placement.h", "kernel_attrs.h", "serve_common.cuh",
           "serve_attn.cuh", "serve_attn_rows.cuh", "serve_attn_rows8.cuh", "serve_tc.cuh"]
PUBLIC_HEADERS = ["rra.h", "rra_probe.h", "rra_static.h", "rra_device.cuh", "rra_serve.h"]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--expt-relaxed-constexpr", "-I" + INCLUDE, "-I" + CSRC]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build librra.so")
    return path


def _newest(files) -> float:
    return max(os.path.getmtime(f) for f in [*files, os.path.abspath(__file__)])


def _library_inputs() -> list:
    return [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + [os.path.join(INCLUDE, f) for f in PUBLIC_HEADERS]


def _torch() -> str:
    """What of the installed torch _serve.so depends on; empty if there is none with CUDA (found without importing it)."""
    try:
        spec = importlib.util.find_spec("torch")
    except (ImportError, ValueError):
        spec = None
    if spec is None or not spec.submodule_search_locations:
        return ""
    at = spec.submodule_search_locations[0]
    try:
        text = open(os.path.join(at, "version.py")).read()
    except OSError:
        return ""
    found = dict(re.findall(r"^(__version__|cuda)\b[^=\n]*= *'([^']*)'", text, flags=re.M))
    return "%s %s %s %s" % (at, found.get("__version__"), found["cuda"], sys.version) if "cuda" in found else ""


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


def _native_fresh(torch: str) -> bool:
    inputs = [os.path.join(CSRC, "serve_bind.cpp")] + [os.path.join(INCLUDE, f) for f in ("rra.h", "rra_serve.h")]
    if not (os.path.exists(NATIVE) and os.path.exists(NATIVE_STAMP) and os.path.getmtime(NATIVE) >= _newest(inputs)):
        return False
    return open(NATIVE_STAMP).read() == torch


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile and link; returns the path of librra.so.  Skips work when the
    library is newer than every source.  Where torch is installed, its binding
    _serve.so is built next to it, again if it is another torch or Python; what
    goes wrong there is raised once librra.so is in place."""
    torch = _torch()
    library = force or not (os.path.exists(LIB) and os.path.getmtime(LIB) >= _newest(_library_inputs()))
    binding = torch != "" and (force or not _native_fresh(torch))
    procs = []

    def start(name, cmd):
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        procs.append((name, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))

    def finish(some):
        """Waits for all of them; raises what went wrong."""
        errors = []
        for name, p in some:
            text = p.communicate()[0].decode(errors="replace")
            if p.returncode != 0:
                errors.append("%s:\n%s" % (name, text))
            elif verbose and text.strip():
                print(text, file=sys.stderr)
        if errors:
            raise RuntimeError("compilation failed\n" + "\n".join(errors))

    native = NATIVE + ".tmp%d" % os.getpid()
    os.makedirs(BUILD, exist_ok=True)
    try:
        if library:
            cc, objs = nvcc(), []
            for src in SOURCES:
                objs.append(os.path.join(BUILD, os.path.splitext(src)[0] + ".o"))
                start(src, [cc, *ARCH, *FLAGS, *extra_flags, "-c", os.path.join(CSRC, src), "-o", objs[-1]])
        units = list(procs)
        command = None
        if binding:
            try:
                command = _native_command(native)
                start("serve_bind.cpp", command)
            except Exception as e:  # noqa: BLE001  a torch that does not import: said below
                command = e
        if library:
            finish(units)
            tmp = LIB + ".tmp%d" % os.getpid()
            p = subprocess.run([cc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs], stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
            if p.returncode != 0:
                raise RuntimeError("link failed:\n" + p.stdout.decode(errors="replace"))
            os.replace(tmp, LIB)
        if isinstance(command, Exception):
            raise RuntimeError("librra.so is built, its binding for torch is not: %s" % command) from command
        finish(procs[len(units):])
    finally:
        for _, p in procs:
            if p.returncode is None:
                p.communicate()
    if binding:
        os.replace(native, NATIVE)
        with open(NATIVE_STAMP, "w") as f:
            f.write(torch)
    return LIB


if __name__ == "__main__":
    force = "--force" in sys.argv
    print(build(force=force, verbose=True))
