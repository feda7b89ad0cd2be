"""Build the in-tree CUDA library ``_lib/libpagedkv.so`` for sm_103a with nvcc,
and ``_lib/_pagedkv_binding.so``, the Python module of the calls whose host cost
shows, with the host compiler against torch's headers.

One object per translation unit, compiled in parallel, then one shared link.
The CUDA runtime is linked statically; the driver API entry point for TMA
descriptors is fetched at run time, so the library needs only libcuda.
"""

from __future__ import annotations

import glob
import importlib.util
import os
import shutil
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_DIR = os.path.join(PKG, "_lib")
LIB_PATH = os.path.join(LIB_DIR, "libpagedkv.so")
BINDING_PATH = os.path.join(LIB_DIR, "_pagedkv_binding.so")
BINDING_SRC = os.path.join(CSRC, "torch_binding.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA library cannot be built")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs():
    return sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + \
        sorted(glob.glob(os.path.join(INCLUDE, "*.h"))) + [BINDING_SRC, os.path.abspath(__file__)]


def is_stale() -> bool:
    if not os.path.exists(LIB_PATH) or not os.path.exists(BINDING_PATH):
        return True
    t = min(os.path.getmtime(LIB_PATH), os.path.getmtime(BINDING_PATH))
    return any(os.path.getmtime(f) > t for f in _inputs())


def _compile_binding(nvcc: str) -> str:
    """Object file of the Python module (torch's headers, no CUDA code)."""
    cxx = shutil.which("g++") or shutil.which("c++")
    spec = importlib.util.find_spec("torch")
    if cxx is None or spec is None:
        raise RuntimeError("the Python module needs a C++ compiler and torch")
    torch_inc = os.path.join(spec.submodule_search_locations[0], "include")
    cuda_inc = os.path.join(os.path.dirname(os.path.dirname(nvcc)), "include")
    obj = os.path.join(LIB_DIR, "obj_binding.o")
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-I", INCLUDE]
    for d in (torch_inc, os.path.join(torch_inc, "torch", "csrc", "api", "include"),
              sysconfig.get_paths()["include"], cuda_inc):
        cmd += ["-isystem", d]
    r = subprocess.run(cmd + ["-c", BINDING_SRC, "-o", obj], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cxx} failed on {os.path.basename(BINDING_SRC)}:\n{r.stderr[-4000:]}")
    return obj


def _link_binding(obj: str) -> None:
    spec = importlib.util.find_spec("torch")
    torch_lib = os.path.join(spec.submodule_search_locations[0], "lib")
    tmp = BINDING_PATH + f".tmp{os.getpid()}"
    r = subprocess.run([shutil.which("g++") or shutil.which("c++"), "-shared", obj, "-o", tmp,
                        "-L", LIB_DIR, "-lpagedkv", "-Wl,-rpath,$ORIGIN", "-L", torch_lib, "-lc10",
                        "-lc10_cuda", "-ltorch", "-ltorch_cpu", "-ltorch_python"],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"linking {os.path.basename(BINDING_PATH)} failed:\n{r.stderr}")
    os.replace(tmp, BINDING_PATH)


def build(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    """Compile and link if the library is missing or older than its sources."""
    if not force and not is_stale():
        return LIB_PATH
    nvcc = _nvcc()
    obj_dir = os.path.join(LIB_DIR, "obj")
    os.makedirs(obj_dir, exist_ok=True)
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++20", "-Xcompiler", "-fPIC",
                    "-I", INCLUDE, "-I", CSRC] + list(extra_flags or [])
    if verbose:
        flags += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(obj_dir, os.path.basename(src)[:-3] + ".o")
        r = subprocess.run([nvcc] + flags + ["-c", src, "-o", obj], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with ThreadPoolExecutor(max_workers=min(16, os.cpu_count() or 1)) as ex:
        binding = ex.submit(_compile_binding, nvcc)
        results = list(ex.map(compile_one, sources()))
        binding_obj = binding.result()
    if verbose:
        for _, log in results:
            print(log)
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    r = subprocess.run([nvcc] + ARCH + ["-shared", "-o", tmp] + [o for o, _ in results],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    _link_binding(binding_obj)
    return LIB_PATH


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
