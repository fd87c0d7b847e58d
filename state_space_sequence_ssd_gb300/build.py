"""Build the sm_103a shared library in-tree: state_space_sequence_ssd_gb300/_build/libssd_gb300.so.

Each csrc/*.cu is compiled to an object in parallel with
``nvcc -gencode arch=compute_103a,code=sm_103a`` and linked (static cudart)
into one shared library with a plain C ABI (include/ssd.h).  Beside it,
csrc/layer_binding.cpp becomes ssd_layer_binding.so, the Python module that
marshals the layer operators' calls (host code against torch's headers).  The
library needs no torch: it is built all the same where there is none, and before
an error of the binding is raised.

    python -m state_space_sequence_ssd_gb300.build [--force] [--verbose-ptxas]
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libssd_gb300.so")
BINDING = os.path.join(BUILD, "ssd_layer_binding.so")
BINDING_SRC = os.path.join(CSRC, "layer_binding.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the SSD library")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + [os.path.join(ROOT, "include", "ssd.h")]


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(p) > t for p in _deps())


def _torch_dir() -> str | None:
    """The folder of the torch that would be imported (without importing it)."""
    spec = importlib.util.find_spec("torch")
    return None if spec is None or spec.origin is None else os.path.dirname(spec.origin)


def _binding_lacks() -> str | None:
    """What is missing here to build the binding, if anything."""
    torch_dir = _torch_dir()
    if torch_dir is None:
        return "torch"
    for header in (os.path.join(torch_dir, "include", "ATen", "ATen.h"), os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        if not os.path.exists(header):
            return header
    return None if shutil.which("g++") else "g++"


def _made_for() -> str:
    """The torch and the Python that a binding belongs to."""
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        return f"{sysconfig.get_config_var('SOABI')}\n{f.read()}"


def _binding_stale() -> bool:
    stamp = BINDING + ".made_for"
    if not os.path.exists(BINDING) or not os.path.exists(stamp):
        return True
    with open(stamp) as f:
        if f.read() != _made_for():
            return True
    t = os.path.getmtime(BINDING)
    return any(os.path.getmtime(p) > t for p in (BINDING_SRC, os.path.join(ROOT, "include", "ssd.h")))


def _compile_binding() -> str:
    import torch
    torch_dir = _torch_dir()
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    includes = [os.path.join(ROOT, "include"), sysconfig.get_paths()["include"], os.path.join(cuda, "include"),
                os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include", "torch", "csrc", "api", "include")]
    obj = os.path.join(BUILD, "layer_binding.o")
    r = subprocess.run(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
                        f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                        *(f"-I{p}" for p in includes), "-c", BINDING_SRC, "-o", obj], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {BINDING_SRC}:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_binding(obj: str) -> None:
    tmp = BINDING + f".tmp{os.getpid()}"
    libs = os.path.join(_torch_dir(), "lib")
    r = subprocess.run(["g++", "-shared", "-o", tmp, obj, f"-L{BUILD}", "-l:libssd_gb300.so", "-Wl,-rpath,$ORIGIN", f"-L{libs}",
                        "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10"], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    with open(BINDING + ".made_for", "w") as f:
        f.write(_made_for())


def build(force: bool = False, verbose_ptxas: bool = False, jobs: int | None = None) -> str:
    stale, lacks = force or verbose_ptxas or _stale(), _binding_lacks()
    binding_stale = lacks is None and (force or _binding_stale())
    os.makedirs(BUILD, exist_ok=True)
    if lacks is not None and not os.path.exists(BINDING):
        warnings.warn(f"the layer operators' Python binding is not built: {lacks} is missing here")
    if not stale:
        if binding_stale:
            _link_binding(_compile_binding())
        return LIB
    nvcc = _nvcc()
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
                    "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]
    if verbose_ptxas:
        flags += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        r = subprocess.run([nvcc, *flags, "-c", src, "-o", obj], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=jobs or min(os.cpu_count() or 8, len(srcs) + 1)) as ex:
        binding = ex.submit(_compile_binding) if lacks is None else None  # host code, beside the kernels
        results = list(ex.map(compile_one, srcs))
    if verbose_ptxas:
        for _, log in results:
            if log.strip():
                print(log)
    tmp = LIB + f".tmp{os.getpid()}"
    r = subprocess.run([nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp] + [o for o, _ in results],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if binding is not None:
        _link_binding(binding.result())
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose-ptxas", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose_ptxas=a.verbose_ptxas))
