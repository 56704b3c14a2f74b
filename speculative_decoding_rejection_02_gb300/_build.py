"""Build of the verifier's CUDA library (nvcc, sm_103a only).

``build()`` compiles ``csrc/spec_verify.cu`` (the verifier),
``csrc/spec_cache.cu`` (the paged cache) and ``csrc/spec_sparse.cu`` (its sparse
attention and eviction), one translation unit each that includes its kernels, into ``_lib/libspecverify.so`` inside the package, and
``csrc/cache_binding.cpp`` (the paged cache's calls on torch tensors) into the
Python module ``_lib/_cache_binding.so``.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import re
import shutil
import subprocess
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB_DIR = os.path.join(PKG, "_lib")
LIB_PATH = os.path.join(LIB_DIR, "libspecverify.so")
BINDING_PATH = os.path.join(LIB_DIR, "_cache_binding.so")
HEADERS = [os.path.join(ROOT, "include", h)
           for h in ("spec_verify.h", "spec_cache.h", "spec_sparse.h")]
UNITS = ("spec_verify", "spec_cache", "spec_sparse")

NVCC_FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC",
]


def _newest(*patterns):
    files = [f for p in patterns for f in glob.glob(os.path.join(CSRC, p))]
    return max(os.path.getmtime(f) for f in files + HEADERS)


def _stale(path, *patterns):
    return not os.path.exists(path) or os.path.getmtime(path) < _newest(*patterns)


def _nvcc():
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _torch_dir():
    """Where torch is installed, without importing it; None where it is not."""
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec else None


def torch_version():
    """Of the torch that is installed, without importing it where its version.py tells."""
    path = os.path.join(_torch_dir(), "version.py")
    if os.path.exists(path):
        with open(path) as f:
            found = re.search(r"""^__version__\s*=\s*['"](.+?)['"]""", f.read(), re.M)
        if found:
            return found.group(1)
    import torch
    return str(torch.__version__)


def binding_torch():
    """The torch version that the Python module was built for; None without a note of it."""
    try:
        with open(BINDING_PATH + ".torch") as f:
            return f.read()
    except FileNotFoundError:
        return None


def _binding_lacks():
    """What the Python module cannot be built without, or None where all is there."""
    torch_dir = _torch_dir()
    if torch_dir is None:
        return "torch is not installed"
    if not os.path.exists(os.path.join(torch_dir, "include", "ATen", "ATen.h")):
        return "torch's headers are not installed"
    if shutil.which("g++") is None:
        return "there is no g++"
    return None


def _binding_command(out):
    """The host compiler's command for the Python module (torch's headers, no torch import)."""
    torch_dir = _torch_dir()
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
    """Compile what is missing or older than its sources. The library needs nvcc alone: where
    the Python module cannot be built (a warning says why) the cache's calls on tensors raise,
    and all else works."""
    os.makedirs(LIB_DIR, exist_ok=True)
    tag = f".tmp{os.getpid()}"
    extra = ["-Xptxas=-v"] if verbose else []
    objs, jobs, binding = [], {}, None  # jobs: every compiler that was started, by source
    if force or _stale(LIB_PATH, "*.cu", "*.cuh"):
        objs = [os.path.join(LIB_DIR, u + tag + ".o") for u in UNITS]
        for u, o in zip(UNITS, objs):
            jobs[u + ".cu"] = subprocess.Popen([_nvcc(), *NVCC_FLAGS, *extra, "-c", "-o", o,
                                                os.path.join(CSRC, u + ".cu")])
    lacks = _binding_lacks()
    if lacks:
        warnings.warn(f"the paged cache's Python module is not built: {lacks}")
    elif force or _stale(BINDING_PATH, "*.cpp") or binding_torch() != torch_version():
        binding = BINDING_PATH + tag
        jobs["cache_binding.cpp"] = subprocess.Popen(_binding_command(binding))
    failed = [n for n, p in jobs.items() if p.wait() != 0]
    try:
        if objs and not any(n.endswith(".cu") for n in failed):
            subprocess.run([_nvcc(), *NVCC_FLAGS, "-shared", "-o", LIB_PATH + tag, *objs],
                           check=True)
            os.replace(LIB_PATH + tag, LIB_PATH)
        if binding and "cache_binding.cpp" not in failed:
            os.replace(binding, BINDING_PATH)
            with open(binding, "w") as f:
                f.write(torch_version())
            os.replace(binding, BINDING_PATH + ".torch")
    finally:
        for x in [*objs, binding, LIB_PATH + tag]:
            if x and os.path.exists(x):
                os.remove(x)
    if failed:
        raise RuntimeError("the compiler failed on " + ", ".join(failed))
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose=True))
