"""The extension module with the prompt calls' checks is a convenience: no call needs it, and one
that was built for another torch is neither used nor left as it is."""

import os
import shutil
import subprocess
import sys

import pytest

from mla_latent_kv_45_b200 import _lib as L
from mla_latent_kv_45_b200 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

USE = """
import warnings
import torch
from mla_latent_kv_45_b200 import _lib as L
%s
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    L.lib()
assert L._marshal is None
assert any("_marshal" in str(w.message) and %r in str(w.message) for w in seen), seen
# decode and prompt calls reach the library, and the checks in Python say what is wrong
assert L.mla_workspace_size(L.Dims(128, 512, 64, 128, 128, 64), 4, 5120, 0, 0) > 0
d = L.Dims(2, 512, 64, 128, 128, 64)
assert L.mla_prompt_workspace_size(d, 1, 8) > 0
z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
cu = torch.tensor([0, 3], dtype=torch.int32)
cache = L.PagedCache(z(2, 64, 576), torch.zeros(1, 2, dtype=torch.int32), None)
for f in (lambda: L.mla_prompt_attn(d, z(3, 2, 128), z(3, 2, 64), z(3, 2, 128), z(3, 64), z(3, 2, 128),
                                    cu, cu, z(3, 2, 128), None, z(8)),
          lambda: L.mla_prompt_append(d, cache, z(3, 576), z(512), cu, ws=z(8)),
          lambda: L.mla_cache_gather(d, cache, cu, None, z(3, 576), z(8))):
    try:
        f()
    except ValueError as e:
        assert "mla_" in str(e)
    else:
        raise AssertionError("tensors of the host were taken")
print("fine")
"""


@pytest.fixture(scope="module")
def built():
    build.build()
    L.lib()


def package(tmp_path, module):
    at = tmp_path / "mla_latent_kv_45_b200"
    at.mkdir()
    for f in os.listdir(build.HERE):
        if f.endswith(".py") or f == os.path.basename(build.LIB) or module and f.startswith("_marshal"):
            shutil.copy2(os.path.join(build.HERE, f), at / f)
    return tmp_path


def use(where, code):
    r = subprocess.run([sys.executable, "-c", code], cwd=where, capture_output=True, text=True,
                       env={**os.environ, "PYTHONPATH": str(where)}, timeout=300)
    assert r.returncode == 0 and r.stdout.endswith("fine\n"), r.stdout + r.stderr


def test_every_call_works_without_the_module(built, tmp_path):
    use(package(tmp_path, False), USE % ("", "_marshal"))


def test_a_module_that_cannot_be_loaded_is_not_used(built, tmp_path):
    where = package(tmp_path, False)
    (where / "mla_latent_kv_45_b200" / os.path.basename(build.MARSHAL)).write_bytes(b"no module")
    use(where, USE % ("", "_marshal"))


def test_a_module_for_another_torch_is_not_used(built, tmp_path):
    use(package(tmp_path, True), USE % ("L.torch_build = lambda: 'another'", "this is another"))


def test_a_module_for_another_torch_is_built_again(built, monkeypatch, tmp_path):
    assert build.up_to_date()
    made = []
    monkeypatch.setattr(build, "_build_marshal", lambda: made.append(1))
    monkeypatch.setattr(build, "_compile", lambda *a: pytest.fail("the library is newer"))
    build.build()
    assert not made
    monkeypatch.setattr(L, "torch_build", lambda: "another")
    assert not build.up_to_date()
    build.build()
    assert made == [1]
    monkeypatch.undo()
    monkeypatch.setattr(build, "STAMP", str(tmp_path / "none"))
    assert not build.up_to_date()


def test_a_machine_that_cannot_compile_the_module_gets_the_library(built, monkeypatch, capsys):
    def fails():
        raise RuntimeError("no headers")

    monkeypatch.setattr(build, "_build_marshal", fails)
    monkeypatch.setattr(build, "marshal_up_to_date", lambda: False)
    assert build.build() == build.LIB
    assert "no headers" in capsys.readouterr().err
