"""Build libpa_gb300.so in-tree with nvcc for sm_103a (GB300).

Each translation unit compiles in parallel into ``_build/``; the objects are
linked into ``libpa_gb300.so`` next to this file.  Beside it, with the host compiler, the
binding's descriptor code (``_marshal.so``, csrc/pa_marshal.cpp).  Rebuilds only when a source or
header is newer than the library.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libpa_gb300.so")
# (the slowest to compile first)
SOURCES = ["pa_decode_mma_fp4.cu", "pa_decode_mma16.cu", "pa_decode_mma_fp8.cu", "pa_decode_window_fp4.cu",
           "pa_rotary_f32.cu", "pa_decode_window_16.cu", "pa_decode_window_fp8.cu", "pa_rotary_bf16.cu", "pa_rotary_f16.cu",
           "pa_chunk_window.cu", "pa_chunk_mma16.cu", "pa_fp4.cu", "pa_decode.cu", "pa_evict.cu", "pa_write.cu", "pa_api.cu",
           "pa_noalloc.cu", "pa_blocks.cu"]
MARSHAL_SOURCE = os.path.join(CSRC, "pa_marshal.cpp")
MARSHAL = os.path.join(HERE, "_marshal.so")
NO_MARSHAL = os.path.join(BUILD, "no_marshal")  # it could not be compiled here
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVFLAGS = ["-O3", "-std=c++17", "-lineinfo", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC",
           "-Xcompiler", "-fvisibility=hidden", "-Xptxas", "-warn-spills"]


def _nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpa_gb300.so")


def _inputs():
    return ([os.path.join(CSRC, s) for s in SOURCES] + glob.glob(os.path.join(CSRC, "*.cuh"))
            + glob.glob(os.path.join(CSRC, "*.h"))
            + [MARSHAL_SOURCE, os.path.join(ROOT, "include", "pa.h"), __file__])


def stale() -> bool:
    if not os.path.exists(LIB) or not (os.path.exists(MARSHAL) or os.path.exists(NO_MARSHAL)):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(f) > t for f in _inputs())


def _build_marshal() -> None:
    """_marshal.so against the installed torch.  Without it the binding describes tensors in Python, so a
    machine without torch's headers still builds."""
    import sysconfig

    import torch
    base = os.path.dirname(torch.__file__)
    tmp = MARSHAL + ".%d.tmp" % os.getpid()
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI), '-DPA_TORCH="%s"' % torch.__version__,
           "-I", os.path.join(base, "include"), "-I", os.path.join(base, "include", "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"], MARSHAL_SOURCE, "-o", tmp, "-L", os.path.join(base, "lib"),
           "-lc10", "-ltorch_cpu", "-ltorch_python"]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
        failed = r.stdout + r.stderr if r.returncode != 0 else None
    except OSError as e:  # no such compiler
        failed = str(e)
    if failed is not None:
        open(NO_MARSHAL, "w").close()
        if os.path.exists(MARSHAL):  # (of an earlier source: its descriptors may be others)
            os.remove(MARSHAL)
        sys.stderr.write("pa_marshal.cpp was not compiled (calls take longer on the host):\n%s\n" % failed[-2000:])
        return
    os.replace(tmp, MARSHAL)


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    if not force and not stale():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc, *ARCH, *NVFLAGS, *extra, "-I", os.path.join(ROOT, "include"), "-c",
               os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, " ".join(cmd), r.stdout + r.stderr))
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        marshal = ex.submit(_build_marshal)
        objs = list(ex.map(compile_one, SOURCES))
        marshal.result()
    tmp = LIB + ".%d.tmp" % os.getpid()
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (" ".join(cmd), r.stdout + r.stderr))
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else [])
    print(LIB)
