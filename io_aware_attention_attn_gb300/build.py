"""Build ``libattn_gb300.so`` in-tree with nvcc for sm_103a (no cmake, no torch extension).

Each ``csrc/*.cu`` translation unit is compiled to an object in ``_build/`` in parallel, then
linked into a shared library next to this file.  CUDA's runtime is linked statically, so the
library only needs the NVIDIA driver at run time.

``csrc/py_binding.cpp`` (marshalling of torch tensors for the generation path) is compiled alongside
with the host compiler against torch's and Python's headers.  It is kept up to date by itself: the
library needs neither, is built without them, and does not start over when the binding fails.
The binding fits one torch and one Python; a key beside it says which.

Usage: ``python -m io_aware_attention_attn_gb300.build [--library] [--verbose-ptxas] [--force]``.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libattn_gb300.so")
BINDING = os.path.join(PKG, "_attn_binding.so")
BINDING_SRC = os.path.join(CSRC, "py_binding.cpp")
BINDING_KEY = BINDING + ".key"

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr",
              "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libattn_gb300")


def sources() -> list:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _newer_than_inputs(built: str, files: list) -> bool:
    files = files + [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)] + [os.path.abspath(__file__)]
    return os.path.exists(built) and os.path.getmtime(built) >= max(os.path.getmtime(f) for f in files)


def library_up_to_date() -> bool:
    return _newer_than_inputs(LIB, [os.path.join(CSRC, f) for f in os.listdir(CSRC)
                                    if not f.endswith(".cpp")])


def have_torch() -> bool:
    return importlib.util.find_spec("torch") is not None


def binding_key() -> str:
    """What the binding is compiled against: torch's version and C++ ABI, Python's version, ABI and machine."""
    import torch
    return f"{torch.__version__} {int(torch._C._GLIBCXX_USE_CXX11_ABI)} {sysconfig.get_config_var('EXT_SUFFIX')}"


def binding_matches() -> bool:
    """Whether the binding on disk was built for this torch and this Python."""
    try:
        with open(BINDING_KEY) as f:
            return f.read() == binding_key()
    except FileNotFoundError:
        return False


def binding_up_to_date() -> bool:
    return _newer_than_inputs(BINDING, [BINDING_SRC]) and binding_matches()


def up_to_date() -> bool:
    return library_up_to_date() and (not have_torch() or binding_up_to_date())


def _compile(src: str, verbose_ptxas: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
    if verbose_ptxas:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    if verbose_ptxas:
        sys.stderr.write(r.stderr)
    return obj


def _run(cmd, what: str):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _compile_binding() -> str:
    import torch
    obj = os.path.join(BUILD, "py_binding.o")
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    dirs = [INCLUDE, inc, os.path.join(inc, "torch", "csrc", "api", "include"),
            sysconfig.get_paths()["include"], cuda]
    _run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          *(f for d in dirs for f in ("-isystem" if d is not INCLUDE else "-I", d)),
          "-c", BINDING_SRC, "-o", obj], "compiling py_binding.cpp")
    return obj


def _link_binding(obj: str):
    import torch
    tlib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + ".tmp"
    _run([os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, "-L", PKG, "-l:libattn_gb300.so",
          "-L", tlib, "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10", "-lc10_cuda",
          "-Wl,-rpath,$ORIGIN"], "linking the binding")
    if os.path.exists(BINDING_KEY):
        os.remove(BINDING_KEY)  # at no time beside a binding that it does not describe
    os.replace(tmp, BINDING)
    with open(BINDING_KEY, "w") as f:
        f.write(binding_key())


def build(force: bool = False, verbose_ptxas: bool = False, library_only: bool = False) -> str:
    """Compile and link what is older than its inputs: the library, and the binding where there is a torch
    to build it for.  Returns the library's path."""
    want_lib = force or verbose_ptxas or not library_up_to_date()
    want_binding = not library_only and have_torch() and (force or not binding_up_to_date())
    if not want_lib and not want_binding:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources() if want_lib else []
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        binding = ex.submit(_compile_binding) if want_binding else None
        objs = list(ex.map(lambda s: _compile(s, verbose_ptxas), srcs))
    if want_lib:
        tmp = LIB + ".tmp"
        _run([nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-Xlinker", "-soname=libattn_gb300.so"], "link")
        os.replace(tmp, LIB)
    if want_binding:
        _link_binding(binding.result())
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose-ptxas", action="store_true")
    ap.add_argument("--library", action="store_true", help="without the binding for torch")
    a = ap.parse_args()
    print(build(force=a.force, verbose_ptxas=a.verbose_ptxas, library_only=a.library))
