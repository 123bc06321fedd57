"""Build the CUDA library ``libw4.so`` in-tree with nvcc, for sm_103a only.

Each translation unit compiles in parallel to ``_obj/*.o``; the shared library
links against the shared CUDA runtime (the same one PyTorch loads). A unit is
rebuilt when it or any header is newer than its object file. ``binding.cpp``, the
compiled half of the Python binding, becomes the extension module ``_binding``
against PyTorch's headers and ``libw4.so``.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJ = os.path.join(PKG, "_obj")
LIB = os.path.join(PKG, "libw4.so")
BINDING = os.path.join(PKG, "_binding.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xptxas", "-warn-spills",
         "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libw4.so")
    return path


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _host_flags():
    """g++ flags for the extension module: PyTorch's and CUDA's headers, Python's, and the C++ ABI PyTorch was built with."""
    import sysconfig

    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    dirs = [inc, os.path.join(inc, "torch", "csrc", "api", "include"), cuda, sysconfig.get_paths()["include"], INCLUDE]
    return ["-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"] + \
        [f for d in dirs for f in ("-isystem", d)]


def _run(cmd, what: str, verbose: bool):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def build(verbose: bool = False, extra_flags=None) -> str:
    """Compile every kernel for sm_103a and link ``libw4.so``; return its path."""
    os.makedirs(OBJ, exist_ok=True)
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    headers = _headers()
    cc = nvcc()
    flags = FLAGS + list(extra_flags or [])

    def compile_one(src: str) -> str:
        obj = os.path.join(OBJ, os.path.basename(src)[:-3] + ".o")
        if _stale(obj, [src] + headers) or extra_flags:
            cmd = [cc] + ARCH + flags + ["-c", src, "-o", obj]
            if verbose:
                print(" ".join(cmd), flush=True)
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
            if verbose and (r.stdout or r.stderr):
                print(r.stdout + r.stderr, flush=True)
        return obj

    host_src, host_obj = os.path.join(CSRC, "binding.cpp"), os.path.join(OBJ, "binding.o")

    def compile_host():
        if _stale(host_obj, [host_src] + headers):
            _run(["g++"] + _host_flags() + ["-c", host_src, "-o", host_obj], "g++ on binding.cpp", verbose)

    with cf.ThreadPoolExecutor(max_workers=min(12, os.cpu_count() or 1)) as ex:
        host = ex.submit(compile_host)
        objs = list(ex.map(compile_one, sources))
        host.result()
    if _stale(LIB, objs):
        tmp = LIB + ".tmp"
        cmd = [cc] + ARCH + ["-shared", "-cudart", "shared", "-o", tmp] + objs
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    if _stale(BINDING, [host_obj, LIB]):
        import torch
        tmp = BINDING + ".tmp"
        _run(["g++", "-shared", "-o", tmp, host_obj, "-L", os.path.join(os.path.dirname(torch.__file__), "lib"), "-lc10",
              "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch", "-ltorch_python", "-L", PKG, "-l:libw4.so",
              "-Wl,-rpath,$ORIGIN"], "link of the binding", verbose)
        os.replace(tmp, BINDING)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
