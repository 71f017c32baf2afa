"""Build the CUDA library ``libgdn.so`` in-tree with nvcc, for sm_103a only.

Translation units are compiled in parallel and linked into one shared library
(``_build/libgdn.so`` inside this package).  A rebuild happens only when a
source or header is newer than the library.

Beside it goes ``_build/gdn_torch.so``, a CPython module that does the tensor wrappers'
checks in C++ (g++, against the installed PyTorch's headers); without it they run in Python.
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
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libgdn.so")
TORCH_SRC = os.path.join(CSRC, "gdn_torch.cpp")
TORCH_LIB = os.path.join(BUILD, "gdn_torch.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc_path() -> str:
    p = shutil.which("nvcc")
    if p:
        return p
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libgdn.so")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + [os.path.join(ROOT, "include", "gdn.h")]


def needs_build() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(p) > t for p in _deps() + [TORCH_SRC])


def _compile_torch_module() -> str:
    """Compile gdn_torch.cpp; the object file, or "" where PyTorch's or Python's headers are missing."""
    import sysconfig

    try:
        import torch
        from torch.utils import cpp_extension
    except ImportError:
        return ""
    inc = cpp_extension.include_paths() + [sysconfig.get_paths()["include"], os.path.join(ROOT, "include"),
                                           "/usr/local/cuda/include"]
    obj = os.path.join(BUILD, "gdn_torch.o")
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    r = subprocess.run(["g++", "-O2", "-std=c++17", "-fPIC", "-w", f"-D_GLIBCXX_USE_CXX11_ABI={abi}",
                        *(f"-I{p}" for p in inc), "-c", TORCH_SRC, "-o", obj], capture_output=True, text=True)
    if r.returncode != 0:
        print("gdn_torch.cpp did not compile, the tensor wrappers check in Python:\n" + r.stderr[-2000:])
        return ""
    return obj


def _link_torch_module(obj: str) -> None:
    import torch

    tmp = TORCH_LIB + f".tmp{os.getpid()}"
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    r = subprocess.run(["g++", "-shared", "-o", tmp, obj, f"-L{BUILD}", "-l:libgdn.so", "-Wl,-rpath,$ORIGIN", f"-L{lib}",
                        "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10", "-lc10_cuda"], capture_output=True,
                       text=True)
    if r.returncode != 0:
        print("gdn_torch.so did not link, the tensor wrappers check in Python:\n" + r.stderr[-2000:])
        return
    os.replace(tmp, TORCH_LIB)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    if not force and not needs_build():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = nvcc_path()
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
                    "-I", os.path.join(ROOT, "include"), *extra_flags]
    if verbose:
        flags += ["-Xptxas", "-v"]
    objs = []

    def one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        r = subprocess.run([nvcc, *flags, "-c", src, "-o", obj], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    if os.path.exists(TORCH_LIB):
        os.remove(TORCH_LIB)
    with cf.ThreadPoolExecutor(max_workers=min(16, os.cpu_count() or 1)) as ex:
        torch_obj = ex.submit(_compile_torch_module)
        for obj, log in ex.map(one, sources()):
            objs.append(obj)
            if verbose and log:
                print(log)
    tmp = LIB + f".tmp{os.getpid()}"
    r = subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if torch_obj.result():
        _link_torch_module(torch_obj.result())
    return LIB


if __name__ == "__main__":
    import sys

    print(build(force=True, verbose="-v" in sys.argv))
