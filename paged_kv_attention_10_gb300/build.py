"""Compile the CUDA sources into the in-tree shared library ``libpagedkv.so`` (sm_103a).

Each ``csrc/*.cu`` is compiled in parallel to an object under ``_build/`` and the objects are
linked into one shared library with the CUDA runtime linked statically, so the library loads on
a machine without a GPU (it needs the driver only when a call is made).  ``csrc/binding.cpp``, the
Python binding's checked calls, becomes the extension module ``_checked.so`` against the installed
PyTorch's headers; where that cannot be compiled the binding makes its checks in Python.
"""

from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libpagedkv.so")
BINDING = os.path.join(CSRC, "binding.cpp")
CHECKED = os.path.join(HERE, "_checked.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "pagedkv.h")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-DNDEBUG"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpagedkv.so")
    return cand


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _compile(src: str, verbose_ptxas: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [_nvcc(), *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
    if verbose_ptxas:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    if verbose_ptxas:
        sys.stderr.write(r.stderr)
    return obj


def _newer(target: str, deps) -> bool:
    return os.path.exists(target) and os.path.getmtime(target) >= max(os.path.getmtime(d) for d in deps)


def _compile_binding() -> str:
    """Compile binding.cpp; returns the object, or "" with a note on stderr where it does not compile."""
    import torch

    root = os.path.dirname(torch.__file__)
    obj = os.path.join(BUILD, "binding.o")
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include"), sysconfig.get_paths()["include"]]
    cmd = [shutil.which("c++") or "g++", "-O2", "-std=c++17", "-fPIC", "-DNDEBUG",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DPKV_TORCH="{torch.__version__}"', *(f"-I{d}" for d in inc),
           "-c", BINDING, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(f"binding.cpp did not compile, the binding checks in Python:\n{r.stderr[-2000:]}\n")
        return ""
    return obj


def _link_binding(obj: str) -> None:
    import torch

    tmp = CHECKED + ".tmp"
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = [shutil.which("c++") or "g++", "-shared", "-o", tmp, obj, f"-L{libs}", "-ltorch_python", "-ltorch_cpu",
           "-lc10", "-lc10_cuda", f"-L{HERE}", "-l:libpagedkv.so", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(f"_checked.so did not link, the binding checks in Python:\n{r.stderr[-2000:]}\n")
        return
    os.replace(tmp, CHECKED)


def build(verbose_ptxas: bool = False, force: bool = False) -> str:
    """Build libpagedkv.so and _checked.so if a source or header is newer; return the library's path."""
    os.makedirs(BUILD, exist_ok=True)
    deps = sources() + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cuh")]
    deps.append(HEADER)
    lib_done = not force and _newer(LIB, deps)
    checked_done = not force and _newer(CHECKED, [BINDING, HEADER])
    if lib_done and checked_done:
        return LIB
    srcs = [] if lib_done else sources()
    with cf.ThreadPoolExecutor(max_workers=min(9, len(srcs) + 1)) as ex:
        binding = None if checked_done else ex.submit(_compile_binding)
        objs = list(ex.map(lambda s: _compile(s, verbose_ptxas), srcs))
    if not lib_done:
        _link(objs)
    if binding is not None and binding.result():
        _link_binding(binding.result())
    return LIB


def _link(objs) -> None:
    tmp = LIB + ".tmp"
    cmd = [_nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(verbose_ptxas="-v" in sys.argv, force="-f" in sys.argv))
