"""Builds ``libmla_b200.so`` in-tree with nvcc for sm_100a.

``python -m mla_latent_kv_45_b200.build`` (or ``build()``) compiles every
``csrc/*.cu`` to an object under ``_build/`` and links the shared library next
to this file, and ``csrc/marshal.cpp``, the binding's argument checks, as an extension
module beside it.  Nothing is rebuilt that is newer than its sources; the module, which reads
tensors through the C++ headers of one torch build, also where that is not the torch in use.
The library does not need the module, nor the calls (``_lib.py`` has the same checks in
Python), so a machine that cannot compile it gets a message and the library.
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
STAMP = os.path.join(BUILD_DIR, "marshal.torch")    # the torch that the module was built for

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
            + [os.path.join(ROOT, "include", "mla.h"), __file__])


def _newer(target: str, deps) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(p) <= t for p in deps)


def marshal_up_to_date() -> bool:
    from ._lib import torch_build

    if not _newer(MARSHAL, [MARSHAL_SRC, os.path.join(ROOT, "include", "mla.h"), __file__]):
        return False
    try:
        with open(STAMP) as f:
            return f.read() == torch_build()
    except OSError:
        return False


def up_to_date() -> bool:
    return _newer(LIB, _deps()) and marshal_up_to_date()


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

    from ._lib import torch_build

    tmp = MARSHAL + ".tmp"
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    includes = [sysconfig.get_paths()["include"], os.path.join(ROOT, "include"),
                os.path.join(cuda, "include"), *cpp_extension.include_paths()]
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = [shutil.which("g++") or "c++", "-O2", "-std=c++20", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DMLA_BUILT_FOR="{torch_build()}"',
           *(f for d in includes for f in ("-isystem", d)), MARSHAL_SRC, "-o", tmp, "-L", libs,
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", f"-Wl,-rpath,{libs}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed on {MARSHAL_SRC}:\n{r.stdout}\n{r.stderr}")
    if r.stderr.strip():
        sys.stderr.write(r.stderr)
    os.replace(tmp, MARSHAL)
    with open(STAMP, "w") as f:
        f.write(torch_build())


def build(force: bool = False, extra=()) -> str:
    """Compile and link the library and the module; returns the library's path."""
    anew = force or bool(extra)
    library, module = anew or not _newer(LIB, _deps()), anew or not marshal_up_to_date()
    if not library and not module:
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        marshal = ex.submit(_build_marshal) if module else None
        objs = list(ex.map(lambda s: _compile(s, list(extra)), _sources())) if library else []
    if library:
        _link(objs)
    if marshal:
        try:
            marshal.result()
        except (ImportError, OSError, RuntimeError) as e:
            sys.stderr.write(f"the binding's checks in C++ were not built, those in Python will "
                             f"do: {e}\n")
    return LIB


def _link(objs):
    tmp = LIB + ".tmp"
    # static CUDA runtime; the driver API (tensor-map encoding) is reached
    # through cudaGetDriverEntryPoint, so the library loads on hosts without a GPU
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv,
                extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else ()))
