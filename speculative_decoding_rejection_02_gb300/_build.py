"""Build of the verifier's CUDA library (nvcc, sm_103a only).

``build()`` compiles ``csrc/spec_verify.cu`` (the verifier) and
``csrc/spec_cache.cu`` (the paged cache), one translation unit each that
includes its kernels, into ``_lib/libspecverify.so`` inside the package, and
``csrc/cache_binding.cpp`` (the paged cache's calls on torch tensors) into the
Python module ``_lib/_cache_binding.so``.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB_DIR = os.path.join(PKG, "_lib")
LIB_PATH = os.path.join(LIB_DIR, "libspecverify.so")
BINDING_PATH = os.path.join(LIB_DIR, "_cache_binding.so")
HEADERS = [os.path.join(ROOT, "include", h) for h in ("spec_verify.h", "spec_cache.h")]
UNITS = ("spec_verify", "spec_cache")

NVCC_FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC",
]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(CSRC, "*.cpp")) + HEADERS)


def _nvcc():
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _binding_command(out):
    """The host compiler's command for the Python module (torch's headers, no torch import)."""
    torch_dir = importlib.util.find_spec("torch").submodule_search_locations[0]
    nvcc = _nvcc()
    cuda = os.path.dirname(os.path.dirname(nvcc)) if os.path.sep in nvcc else "/usr/local/cuda"
    dirs = [os.path.join(torch_dir, "include"),
            os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
            os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    return ["g++", "-std=c++17", "-O2", "-fPIC", "-shared", "-o", out,
            os.path.join(CSRC, "cache_binding.cpp"), *[x for d in dirs for x in ("-isystem", d)],
            "-L" + os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch_cuda",
            "-ltorch_cpu", "-lc10_cuda", "-lc10"]


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(LIB_DIR, exist_ok=True)
    if not force and os.path.exists(LIB_PATH) and os.path.exists(BINDING_PATH):
        newest = max(os.path.getmtime(s) for s in _sources())
        if min(os.path.getmtime(LIB_PATH), os.path.getmtime(BINDING_PATH)) >= newest:
            return LIB_PATH
    tag = f".tmp{os.getpid()}"
    objs = [os.path.join(LIB_DIR, u + tag + ".o") for u in UNITS]
    extra = ["-Xptxas=-v"] if verbose else []
    units = [subprocess.Popen([_nvcc(), *NVCC_FLAGS, *extra, "-c", "-o", o,
                               os.path.join(CSRC, u + ".cu")]) for u, o in zip(UNITS, objs)]
    names = [u + ".cu" for u in UNITS] + ["cache_binding.cpp"]
    units.append(subprocess.Popen(_binding_command(BINDING_PATH + tag)))
    failed = [n for n, p in zip(names, units) if p.wait() != 0]  # every compiler is waited for
    try:
        if failed:
            raise RuntimeError("the compiler failed on " + ", ".join(failed))
        subprocess.run([_nvcc(), *NVCC_FLAGS, "-shared", "-o", LIB_PATH + tag, *objs], check=True)
    finally:
        for o in objs:
            if os.path.exists(o):
                os.remove(o)
    os.replace(LIB_PATH + tag, LIB_PATH)
    os.replace(BINDING_PATH + tag, BINDING_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose=True))
