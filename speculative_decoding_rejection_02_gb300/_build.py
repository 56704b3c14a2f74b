"""Build of the verifier's CUDA library (nvcc, sm_103a only).

``build()`` compiles ``csrc/spec_verify.cu`` (the verifier) and
``csrc/spec_cache.cu`` (the paged cache), one translation unit each that
includes its kernels, into ``_lib/libspecverify.so`` inside the package.
"""
from __future__ import annotations

import glob
import os
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB_DIR = os.path.join(PKG, "_lib")
LIB_PATH = os.path.join(LIB_DIR, "libspecverify.so")
HEADERS = [os.path.join(ROOT, "include", h) for h in ("spec_verify.h", "spec_cache.h")]
UNITS = ("spec_verify", "spec_cache")

NVCC_FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC",
]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + HEADERS)


def _nvcc():
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(LIB_DIR, exist_ok=True)
    if not force and os.path.exists(LIB_PATH):
        newest = max(os.path.getmtime(s) for s in _sources())
        if os.path.getmtime(LIB_PATH) >= newest:
            return LIB_PATH
    tag = f".tmp{os.getpid()}"
    objs = [os.path.join(LIB_DIR, u + tag + ".o") for u in UNITS]
    extra = ["-Xptxas=-v"] if verbose else []
    units = [subprocess.Popen([_nvcc(), *NVCC_FLAGS, *extra, "-c", "-o", o,
                               os.path.join(CSRC, u + ".cu")]) for u, o in zip(UNITS, objs)]
    failed = [u for u, p in zip(UNITS, units) if p.wait() != 0]  # every compiler is waited for
    try:
        if failed:
            raise RuntimeError("nvcc failed on " + ", ".join(u + ".cu" for u in failed))
        subprocess.run([_nvcc(), *NVCC_FLAGS, "-shared", "-o", LIB_PATH + tag, *objs], check=True)
    finally:
        for o in objs:
            if os.path.exists(o):
                os.remove(o)
    os.replace(LIB_PATH + tag, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose=True))
