"""A C++ exception inside a library call is caught with the interpreter's lock held again."""

import os
import shutil
import subprocess
import sys

import pytest

from mla_latent_kv_45_b200 import _lib as L
from mla_latent_kv_45_b200 import build

pytestmark = pytest.mark.gpu

USE = """
import ctypes, sys, threading
import torch
from mla_latent_kv_45_b200 import _lib as L
L.lib()
thrower = ctypes.CDLL(sys.argv[1])
at = ctypes.cast(thrower.thrower, ctypes.c_void_p).value
L._marshal.bind(at, at, at)
dims = L.Dims(2, 512, 64, 128, 128, 64)
z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
cu = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
table = torch.zeros(1, 2, dtype=torch.int32, device="cuda")
ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
calls = [lambda: L._marshal.append(dims.c(), z(2, 64, 576), table, z(3, 576), z(512), cu, None, None, None, ws, None),
         lambda: L._marshal.gather(dims.c(), z(2, 64, 576), table, cu, None, z(3, 576), ws, None),
         lambda: L._marshal.attn(dims.c(), z(3, 2, 128), z(3, 2, 64), z(3, 2, 128), z(3, 64), z(3, 2, 128),
                                 cu, cu, z(3, 2, 128), None, ws, None)]
count = ctypes.c_int.in_dll(thrower, "count")
threads = [threading.Thread(target=lambda: [c() for _ in range(200) for c in calls]) for _ in range(3)]
for t in threads:
    t.start()
for t in threads:
    t.join()
assert all(c() is None for c in calls)
assert count.value == 3 * 600 + 3, count.value
print("fine")
"""


def test_exceptions_are_declined_with_the_lock_held(tmp_path):
    build.build()
    L.lib()
    src = tmp_path / "thrower.cpp"
    src.write_text('extern "C" { int count = 0; int thrower() { __atomic_fetch_add(&count, 1, __ATOMIC_SEQ_CST); throw 1; } }')
    so = tmp_path / "thrower.so"
    subprocess.run([shutil.which("g++"), "-shared", "-fPIC", str(src), "-o", str(so)], check=True)
    r = subprocess.run([sys.executable, "-c", USE, str(so)], cwd=build.ROOT, capture_output=True,
                       text=True, timeout=300, env={**os.environ, "PYTHONPATH": build.ROOT})
    assert r.returncode == 0 and r.stdout == "fine\n", r.stdout + r.stderr
