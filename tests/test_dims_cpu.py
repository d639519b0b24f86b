"""Dims is an ordinary dataclass whatever has been called with it."""

import copy
import dataclasses
import pickle
import weakref

import pytest

from mla_latent_kv_45_b200 import _lib as L


def fields(c):
    return [getattr(c, f) for f, _ in c._fields_]


def test_a_struct_belongs_to_whom_it_was_given():
    d = L.Dims(128, 512, 64, 128, 128, 64)
    want = fields(d.c())
    c = d.c()
    c.n_heads = 3
    assert fields(d.c()) == want and fields(d.kept()) == want


def test_the_kept_struct_follows_the_fields():
    d = L.Dims(128, 512, 64, 128, 128, 64)
    k = d.kept()
    assert d.kept() is k and k.n_heads == 128
    d.n_heads = 16
    assert d.kept().n_heads == 16 and d.c().n_heads == 16 and k.n_heads == 128
    d.softmax_scale = 0.5
    assert d.kept().softmax_scale == 0.5


@pytest.mark.parametrize("used", [False, True])
def test_it_is_copied_compared_and_rebuilt_from_its_fields(used):
    d = L.Dims(16, 512, 64, 128, 128, 7, cache_format=L.MLA_CACHE_INT8)
    if used:
        d.kept()
    for other in (copy.copy(d), copy.deepcopy(d), pickle.loads(pickle.dumps(d)), dataclasses.replace(d),
                  L.Dims(**vars(d)), L.Dims(**dataclasses.asdict(d))):
        assert other == d and fields(other.c()) == fields(d.c()) == fields(other.kept())
        other.n_heads = 2
        assert other.kept().n_heads == 2 and d.kept().n_heads == 16 and d.n_heads == 16
    assert set(vars(d)) == {f.name for f in dataclasses.fields(d)}
    assert weakref.ref(d)() is d
    with pytest.raises(AttributeError):
        d.torch_dtype = None
