"""Build the CUDA library in-tree: ``lib/libmuon_adamw_gb300.so``.

Each ``csrc/*.cu`` file is compiled by nvcc for sm_103a only
(``-gencode arch=compute_103a,code=sm_103a``) in parallel, then linked with
the static CUDA runtime into one shared library. The library depends on
nothing but the CUDA driver at run time (resolved lazily, so it also loads
on a machine without a GPU). Rebuilds only when a source or header changed.

``csrc/torch_ops.cpp``, the operators over torch tensors, is host code: g++
compiles it against the installed torch into the extension module
``lib/_torch_ops.so``, which links the library above. The library needs
neither: without torch the module is left out, and where it fails to build
the library is there all the same.
"""
from __future__ import annotations

import hashlib
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor
from typing import Optional

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
TORCH_OPS = "torch_ops.cpp"
CXX_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-I", INCLUDE]


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


def _hash(h, *paths: str) -> None:
    for path in paths:
        h.update(os.path.basename(path).encode())
        with open(path, "rb") as fh:
            h.update(fh.read())


def _digest() -> str:
    """Of what the library is made from."""
    h = hashlib.sha256()
    for d in (CSRC, INCLUDE):
        _hash(h, *(os.path.join(d, f) for f in sorted(os.listdir(d)) if f.endswith((".cu", ".cuh", ".h"))))
    h.update(" ".join(ARCH + NVCC_FLAGS).encode())
    h.update(os.uname().machine.encode())
    return h.hexdigest()


def _torch_dir() -> Optional[str]:
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def _torch_ops_digest(torch_dir: str) -> str:
    """Of what the extension module is made from: it calls the library through the public header alone."""
    h = hashlib.sha256()
    _hash(h, os.path.join(CSRC, TORCH_OPS), os.path.join(INCLUDE, "muon_adamw.h"), os.path.join(torch_dir, "version.py"))
    h.update(" ".join([torch_dir, sys.version, *CXX_FLAGS]).encode())
    h.update(os.uname().machine.encode())
    return h.hexdigest()


def _stamped(path: str, digest: str) -> bool:
    stamp = path + ".sha256"
    if not os.path.exists(path) or not os.path.exists(stamp):
        return False
    with open(stamp) as fh:
        return fh.read().strip() == digest


def _run(what: str, cmd) -> subprocess.CompletedProcess:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what}:\n{r.stdout}\n{r.stderr}")
    return r


def _link(path: str, digest: str, cmd) -> None:
    """`cmd` with its output in place of {}, moved to `path` and stamped."""
    tmp = path + ".tmp"
    _run(f"link of {os.path.basename(path)} failed", [tmp if c == "{}" else c for c in cmd])
    os.replace(tmp, path)
    with open(path + ".sha256", "w") as fh:
        fh.write(digest)


def is_stale() -> bool:
    """The library is missing or older than its sources."""
    return not _stamped(lib_path(), _digest())


def torch_ops_stale() -> bool:
    """torch is installed and the extension module is missing, or older than its source or than torch."""
    torch_dir = _torch_dir()
    return torch_dir is not None and not _stamped(torch_ops_path(), _torch_ops_digest(torch_dir))


def torch_ops_problem() -> str:
    """Why the last build left no extension module ("": it did, or there is no torch)."""
    path = torch_ops_path() + ".problem"
    if not os.path.exists(path):
        return ""
    with open(path) as fh:
        return fh.read()


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link what is stale; return the library's path. A failure of
    the extension module alone is a warning: the library does not need it, and
    importing the operators raises with the reason."""
    library, module = force or is_stale(), torch_ops_stale() or (force and _torch_dir() is not None)
    if not library and not module:
        return lib_path()
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    srcs = _sources() if library else []

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, src[:-3] + ".o")
        r = _run(f"nvcc failed on {src}", [nvcc, *ARCH, *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj])
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, file=sys.stderr)
        return obj

    def compile_torch_ops() -> str:
        obj = os.path.join(BUILD, "torch_ops.o")
        torch_include = os.path.join(_torch_dir(), "include")
        cmd = ["g++", *CXX_FLAGS]
        for d in (torch_include, os.path.join(torch_include, "torch", "csrc", "api", "include"),
                  sysconfig.get_paths()["include"],
                  os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")):
            cmd += ["-isystem", d]
        _run(f"g++ failed on {TORCH_OPS}", [*cmd, "-c", os.path.join(CSRC, TORCH_OPS), "-o", obj])
        return obj

    if module:  # one that no longer fits is not to be loaded, whatever happens now
        for path in (torch_ops_path(), torch_ops_path() + ".sha256", torch_ops_path() + ".problem"):
            if os.path.exists(path):
                os.remove(path)
    with ThreadPoolExecutor(max(1, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        torch_obj = ex.submit(compile_torch_ops) if module else None
        objs = list(ex.map(compile_one, srcs))
    if library:
        _link(lib_path(), _digest(),
              [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", "{}", *objs, "-ldl", "-lpthread", "-lrt"])
    if module:
        try:
            _link(torch_ops_path(), _torch_ops_digest(_torch_dir()),
                  ["g++", "-shared", "-o", "{}", torch_obj.result(), "-L", LIBDIR, f"-l:{LIBNAME}", "-L",
                   os.path.join(_torch_dir(), "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda",
                   "-ltorch_python", "-Wl,-rpath,$ORIGIN"])
        except (RuntimeError, OSError) as e:  # OSError: no g++ at all
            with open(torch_ops_path() + ".problem", "w") as fh:
                fh.write(str(e))
            warnings.warn(f"the operators over torch tensors were not built: {e}", RuntimeWarning, stacklevel=2)
    return lib_path()


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
