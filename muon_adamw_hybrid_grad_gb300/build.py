"""Build the CUDA library in-tree: ``lib/libmuon_adamw_gb300.so``.

Each ``csrc/*.cu`` file is compiled by nvcc for sm_103a only
(``-gencode arch=compute_103a,code=sm_103a``) in parallel, then linked with
the static CUDA runtime into one shared library. The library depends on
nothing but the CUDA driver at run time (resolved lazily, so it also loads
on a machine without a GPU). Rebuilds only when a source or header changed.

``csrc/torch_ops.cpp``, the operators over torch tensors, is host code: g++
compiles it against the installed torch into the extension module
``lib/_torch_ops.so``, which links the library above.
"""
from __future__ import annotations

import hashlib
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIBDIR = os.path.join(PKG, "lib")
LIBNAME = "libmuon_adamw_gb300.so"
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "-I", INCLUDE, "-I", CSRC]


def lib_path() -> str:
    return os.path.join(LIBDIR, LIBNAME)


def torch_ops_path() -> str:
    return os.path.join(LIBDIR, "_torch_ops.so")


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")


def _sources():
    return sorted(f for f in os.listdir(CSRC) if f.endswith(".cu"))


def _digest() -> str:
    h = hashlib.sha256()
    for d in (CSRC, INCLUDE):
        for f in sorted(os.listdir(d)):
            if f.endswith((".cu", ".cuh", ".h", ".cpp")):
                h.update(f.encode())
                with open(os.path.join(d, f), "rb") as fh:
                    h.update(fh.read())
    h.update(" ".join(ARCH + NVCC_FLAGS).encode())
    h.update(os.uname().machine.encode())
    h.update((sys.version + importlib.metadata.version("torch")).encode())
    return h.hexdigest()


def is_stale() -> bool:
    stamp = os.path.join(LIBDIR, LIBNAME + ".sha256")
    if not os.path.exists(lib_path()) or not os.path.exists(torch_ops_path()) or not os.path.exists(stamp):
        return True
    with open(stamp) as fh:
        return fh.read().strip() != _digest()


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link the library if needed; return its path."""
    if not force and not is_stale():
        return lib_path()
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    srcs = _sources()

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, src[:-3] + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, file=sys.stderr)
        return obj

    def compile_torch_ops() -> str:
        obj = os.path.join(BUILD, "torch_ops.o")
        torch_dir = os.path.dirname(importlib.util.find_spec("torch").origin)
        cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
        system = [os.path.join(torch_dir, "include"),
                  os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
                  sysconfig.get_paths()["include"], cuda]
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-I", INCLUDE]
        for d in system:
            cmd += ["-isystem", d]
        r = subprocess.run(cmd + ["-c", os.path.join(CSRC, "torch_ops.cpp"), "-o", obj], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed on torch_ops.cpp:\n{r.stdout}\n{r.stderr}")
        return obj

    with ThreadPoolExecutor(max(1, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        torch_obj = ex.submit(compile_torch_ops)
        objs = list(ex.map(compile_one, srcs))
        torch_obj = torch_obj.result()
    tmp = lib_path() + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs, "-ldl", "-lpthread", "-lrt"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib_path())
    torch_lib = os.path.join(os.path.dirname(importlib.util.find_spec("torch").origin), "lib")
    tmp = torch_ops_path() + ".tmp"
    cmd = ["g++", "-shared", "-o", tmp, torch_obj, "-L", LIBDIR, f"-l:{LIBNAME}", "-L", torch_lib, "-lc10", "-lc10_cuda",
           "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of torch_ops failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, torch_ops_path())
    with open(lib_path() + ".sha256", "w") as fh:
        fh.write(_digest())
    return lib_path()


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
