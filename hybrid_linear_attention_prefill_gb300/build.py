"""Build the CUDA library ``libgdn.so`` in-tree with nvcc, for sm_103a only.

Translation units are compiled in parallel and linked into one shared library
(``_build/libgdn.so`` inside this package).  A rebuild happens only when a
source or header is newer than the library.

Beside it goes ``_build/gdn_torch.<interpreter>.<PyTorch>.so``, a CPython module that does the
tensor functions' checks in C++ (g++, against the installed PyTorch's headers); without it they
run in Python.
"""

from __future__ import annotations

import concurrent.futures as cf
import contextlib
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
    headers = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
    return sources() + headers + [os.path.join(ROOT, "include", "gdn.h")]


def _older(path: str, deps) -> bool:
    if not os.path.exists(path):
        return True
    t = os.path.getmtime(path)
    return any(os.path.getmtime(p) > t for p in deps)


def needs_build() -> bool:
    return _older(LIB, _deps())


def torch_lib() -> str:
    """Path of the gdn_torch module for this interpreter and this PyTorch (whose objects' layout it has compiled in)."""
    import sysconfig

    import torch

    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    return os.path.join(BUILD, f"gdn_torch.{sysconfig.get_config_var('SOABI')}.torch-{torch.__version__}-abi{abi}.so")


def module_needs_build(force: bool = False) -> bool:
    """Whether the gdn_torch module is missing or old; not where there is no PyTorch, nor again after it failed."""
    try:
        path = torch_lib()
    except ImportError:
        return False
    deps = [TORCH_SRC, os.path.join(ROOT, "include", "gdn.h")]
    return force or (_older(path, deps) and _older(path + ".failed", deps))


def _module_step(cmd) -> bool:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        path = torch_lib()
        print(f"{os.path.basename(path)} was not built, the tensor functions check in Python:\n" + r.stderr[-2000:])
        open(path + ".failed", "w").close()
    return r.returncode == 0


def _compile_module(obj: str) -> bool:
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    inc = cpp_extension.include_paths() + [sysconfig.get_paths()["include"], os.path.join(ROOT, "include"),
                                           "/usr/local/cuda/include"]
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    return _module_step(["g++", "-O2", "-std=c++17", "-fPIC", "-w", f"-D_GLIBCXX_USE_CXX11_ABI={abi}",
                         *(f"-I{p}" for p in inc), "-c", TORCH_SRC, "-o", obj])


def _link_module(obj: str) -> None:
    import torch

    path = torch_lib()
    tmp = path + f".tmp{os.getpid()}"
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    if _module_step(["g++", "-shared", "-o", tmp, obj, f"-L{BUILD}", "-l:libgdn.so", "-Wl,-rpath,$ORIGIN", f"-L{lib}",
                     "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10", "-lc10_cuda"]):
        os.replace(tmp, path)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    library, module = force or needs_build(), module_needs_build(force)
    if not library and not module:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    obj = os.path.join(BUILD, f"gdn_torch.{os.getpid()}.o")
    if module:
        with contextlib.suppress(FileNotFoundError):
            os.remove(torch_lib())  # an old one must not stay where the new one does not build
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        compiled = ex.submit(_compile_module, obj) if module else None
        if library:
            _build_library(verbose, extra_flags)
    if module and compiled.result():
        _link_module(obj)
    if os.path.exists(obj):
        os.remove(obj)
    return LIB


def _build_library(verbose: bool, extra_flags) -> None:
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

    with cf.ThreadPoolExecutor(max_workers=min(16, os.cpu_count() or 1)) as ex:
        for obj, log in ex.map(one, sources()):
            objs.append(obj)
            if verbose and log:
                print(log)
    tmp = LIB + f".tmp{os.getpid()}"
    r = subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    import sys

    print(build(force=True, verbose="-v" in sys.argv))
