"""Build librope_qk.so in the package directory with nvcc for sm_103a (GB300)."""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SOURCES = [os.path.join(HERE, "csrc", n) for n in ("rope_qk.cu", "rope_host.cu", "glu.cu", "rope_append.cu",
                                                 "attn.cu", "attn_fwd.cu", "attn_bwd.cu", "attn_decode.cu")]
HEADERS = [os.path.join(ROOT, "include", n) for n in ("rope_qk.h", "glu.h", "paged_kv.h", "attn.h")] + \
          [os.path.join(HERE, "csrc", n) for n in ("fastdiv.cuh", "cos_sin.cuh", "rope_core.cuh", "host_checks.h",
                                                   "paged_checks.h", "attn_internal.h", "tensor_core.cuh", "tensor_map.h")]
LIB_PATH = os.path.join(HERE, "librope_qk.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def flags(verbose_ptxas: bool = False):
    f = ["-O3", "-std=c++17", *ARCH, "-lineinfo", "-Xcompiler", "-fPIC",
         "-I", os.path.join(ROOT, "include")]
    if verbose_ptxas:
        f += ["-Xptxas", "-v"]
    return f


def stale() -> bool:
    if not os.path.exists(LIB_PATH):
        return True
    t = os.path.getmtime(LIB_PATH)
    return any(os.path.getmtime(p) > t for p in SOURCES + HEADERS)


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compile the CUDA library if it is missing or older than its sources."""
    if force or verbose_ptxas or stale():
        tmp = LIB_PATH + ".tmp%d" % os.getpid()
        # one compiler process per source, side by side, then the link
        objs = [tmp + "." + os.path.basename(src) + ".o" for src in SOURCES]
        jobs = [subprocess.Popen([nvcc(), *flags(verbose_ptxas), "-c", src, "-o", obj])
                for src, obj in zip(SOURCES, objs)]
        try:
            for job, src in zip(jobs, SOURCES):
                if job.wait() != 0:
                    raise subprocess.CalledProcessError(job.returncode, "nvcc -c " + src)
            subprocess.check_call([nvcc(), *ARCH, "-shared", "-Xcompiler", "-fPIC", *objs, "-o", tmp])
            os.replace(tmp, LIB_PATH)
        finally:
            for job in jobs:
                job.wait()
            for obj in objs:
                if os.path.exists(obj):
                    os.remove(obj)
    return LIB_PATH


if __name__ == "__main__":
    build(force=True, verbose_ptxas="-v" in sys.argv)
    print(LIB_PATH)
