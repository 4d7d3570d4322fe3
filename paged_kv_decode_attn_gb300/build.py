"""Build ``lib/liboxd.so`` from ``csrc/`` with nvcc for sm_103a.

Sources compile in parallel (one nvcc per translation unit) and link into one
shared library with the CUDA runtime linked statically. The build is skipped
when the library is newer than every source and header.
"""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIBDIR = os.path.join(HERE, "lib")
LIB = os.path.join(LIBDIR, "liboxd.so")
HEADERS = [os.path.join(ROOT, "include", "oxd.h")] + [
    os.path.join(CSRC, h) for h in ("oxd_internal.h", "oxd_merge_row.cuh", "oxd_ptx.cuh",
                                    "oxd_tcgen05.cuh", "oxd_prefill.h", "oxd_host_util.h",
                                    "oxd_e2m1.cuh", "oxd_decode_quant.cuh",
                                    "oxd_decode_quant_state.cuh", "oxd_cache_host.h",
                                    "oxd_window.cuh", "oxd_prefill_window.cuh")]
SOURCES = ["oxd_host.cpp", "oxd_decode.cu", "oxd_decode_wide.cu", "oxd_merge.cu",
           "oxd_noalloc.cu", "oxd_append.cu", "oxd_prefill.cu", "oxd_prefill_narrow.cu",
           "oxd_prefill_window.cu", "oxd_prefill_host.cpp", "oxd_decode_quant.cu", "oxd_decode_quant_wide.cu",
           "oxd_append_axes.cu", "oxd_pages.cu",
           "oxd_quant_host.cpp", "oxd_window_decode.cu", "oxd_window_quant.cu", "oxd_tables.cu",
           "oxd_window_host.cpp"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def common_flags(extra=()):
    return ["-O3", "-std=c++17", *ARCH, "-lineinfo", "-Xcompiler", "-fPIC",
            "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-diag-suppress", "177", *extra]


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, s) for s in SOURCES] + HEADERS + [os.path.abspath(__file__)]
    return any(os.path.getmtime(p) > t for p in deps)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile and link the library if needed; returns its path."""
    if not force and not stale():
        return LIB
    objdir = os.path.join(LIBDIR, "obj")
    os.makedirs(objdir, exist_ok=True)
    procs = []
    objs = []
    for src in SOURCES:
        obj = os.path.join(objdir, src.rsplit(".", 1)[0] + ".o")
        objs.append(obj)
        lang = ["-x", "cu"] if src.endswith(".cu") else []
        cmd = [nvcc(), *common_flags(extra_flags), *lang, "-c", os.path.join(CSRC, src),
               "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE,
                                            stderr=subprocess.STDOUT, text=True)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            failed.append(f"--- {src}\n{out}")
        elif verbose and out:
            print(out, file=sys.stderr)
    if failed:
        raise RuntimeError("nvcc failed:\n" + "\n".join(failed))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stdout)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True,
                extra_flags=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else ()))
