"""Builds ``libmla_b200.so`` in-tree with nvcc for sm_100a.

``python -m mla_latent_kv_45_b200.build`` (or ``build()``) compiles every
``csrc/*.cu`` to an object under ``_build/`` and links the shared library next
to this file, and ``csrc/marshal.cpp``, the binding's argument checks, as an extension
module beside it.  Nothing is rebuilt when both are newer than every source.
"""

from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libmla_b200.so")
MARSHAL = os.path.join(HERE, "_marshal" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
MARSHAL_SRC = os.path.join(HERE, "csrc", "marshal.cpp")
BUILD_DIR = os.path.join(ROOT, "_build")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", os.path.join(ROOT, "include"), "-I", os.path.join(HERE, "csrc")]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found; the CUDA library cannot be built")
    return path


def _sources():
    return sorted(glob.glob(os.path.join(HERE, "csrc", "*.cu")))


def _deps():
    return (_sources() + glob.glob(os.path.join(HERE, "csrc", "*.h"))
            + glob.glob(os.path.join(HERE, "csrc", "*.cuh"))
            + [MARSHAL_SRC, os.path.join(ROOT, "include", "mla.h"), __file__])


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(MARSHAL):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(MARSHAL))
    return all(os.path.getmtime(p) <= t for p in _deps())


def _compile(src: str, extra) -> str:
    obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc(), *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if r.stderr.strip():
        sys.stderr.write(r.stderr)
    return obj


def _build_marshal():
    """The extension module, against the headers and libraries of the torch it runs beside."""
    import torch
    from torch.utils import cpp_extension

    tmp = MARSHAL + ".tmp"
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    includes = [sysconfig.get_paths()["include"], os.path.join(ROOT, "include"),
                os.path.join(cuda, "include"), *cpp_extension.include_paths()]
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = [shutil.which("g++") or "c++", "-O2", "-std=c++20", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f for d in includes for f in ("-isystem", d)), MARSHAL_SRC, "-o", tmp, "-L", libs,
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", f"-Wl,-rpath,{libs}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed on {MARSHAL_SRC}:\n{r.stdout}\n{r.stderr}")
    if r.stderr.strip():
        sys.stderr.write(r.stderr)
    os.replace(tmp, MARSHAL)


def build(force: bool = False, extra=()) -> str:
    """Compile and link the library; returns its path."""
    if not force and not extra and up_to_date():
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        marshal = ex.submit(_build_marshal)
        objs = list(ex.map(lambda s: _compile(s, list(extra)), _sources()))
    tmp = LIB + ".tmp"
    # static CUDA runtime; the driver API (tensor-map encoding) is reached
    # through cudaGetDriverEntryPoint, so the library loads on hosts without a GPU
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    marshal.result()
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv,
                extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else ()))
