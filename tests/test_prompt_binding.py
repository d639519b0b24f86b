"""The prompt calls' two ways through the binding: the checks in C++ decline what they do not
know, and both ways do the same work."""

import pytest
import torch

from mla_latent_kv_45_b200 import _lib as L
from mla_latent_kv_45_b200 import build
import prompt_testlib as T


@pytest.fixture(scope="module")
def marshal():
    build.build()
    L.lib()
    return L._marshal


def test_checks_decline_what_they_do_not_know(marshal):
    dims = T.dims_of(T.V2, 4, torch.bfloat16)
    host = torch.zeros(3, 4, 128, dtype=torch.bfloat16)
    for fn, n in ((marshal.append, 11), (marshal.gather, 8), (marshal.attn, 12)):
        assert fn() is None and fn(*[None] * n) is None
        for other in (None, 3, "x", host, host.view(-1), torch.nn.Module()):
            assert fn(dims.c(), *[other] * (n - 1)) is None
            assert fn(other, *[other] * (n - 1)) is None
        assert fn(b"short", *[host] * (n - 1)) is None
    with pytest.raises(TypeError):
        marshal.bind(1, 2)


def work(kind, stream):
    """Append, gather and attention over one cache; all they wrote."""
    dims = T.dims_of(T.V2, 4, torch.bfloat16, cache=kind)
    new, ctx = [5, 0, 70], [3, 9, 60]
    g = torch.Generator(device="cuda").manual_seed(7)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    if kind == L.MLA_CACHE_INT8:
        pool = torch.zeros(9, 64, L.MLA_INT8_ROW_BYTES, dtype=torch.uint8, device="cuda")
    else:
        pool = torch.zeros(9, 64, 576, dtype=torch.bfloat16, device="cuda")
    cache = L.PagedCache(pool, torch.arange(9, dtype=torch.int32, device="cuda").view(3, 3), None)
    cu_new, cu_all = T.i32(T.offsets(new)), T.i32(T.offsets([a + b for a, b in zip(new, ctx)]))
    n, total = sum(new), sum(new) + sum(ctx)
    x, gamma = r(n, 600)[:, :576], r(512)
    q_rope, q_out = r(n, 4, 64), torch.zeros(n, 4, 64, dtype=torch.bfloat16, device="cuda")
    rows = torch.zeros(total, 576, dtype=torch.bfloat16, device="cuda")
    q_nope, k_nope, v = r(n, 4, 128), r(total, 2, 128), r(total, 2, 128)
    out = torch.zeros(n, 4, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(n, 4, device="cuda")
    ws = T.workspace(dims, 3, total)
    torch.cuda.synchronize()
    L.mla_prompt_append(dims, cache, x, gamma, cu_new, T.i32(ctx), q_rope, q_out, ws, stream=stream)
    L.mla_cache_gather(dims, cache, cu_all, T.i32([0, 0, 0]), rows, ws, stream=stream)
    L.mla_prompt_attn(dims, q_nope, q_out, k_nope, rows[:, 512:], v, cu_new, cu_all, out, lse, ws,
                      stream=stream)
    torch.cuda.synchronize()
    assert L.mla_get_device_error(ws) == 0
    return pool, q_out, rows, out, lse


class Declines:
    append = gather = attn = staticmethod(lambda *a: None)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [L.MLA_CACHE_NATIVE, L.MLA_CACHE_INT8])
def test_both_ways_do_the_same(marshal, monkeypatch, kind):
    taken = []

    class Watched:
        def __getattr__(self, name):
            def f(*a):
                st = getattr(marshal, name)(*a)
                taken.append((name, st))
                return st
            return f

    monkeypatch.setattr(L, "_marshal", Watched())
    side = torch.cuda.Stream()
    got = [work(kind, None), work(kind, side)]
    with torch.cuda.stream(side):
        got.append(work(kind, None))
    assert taken == 3 * [("append", 0), ("gather", 0), ("attn", 0)]
    monkeypatch.setattr(L, "_marshal", Declines)
    for want in (work(kind, None), work(kind, side)):
        for have in got:
            assert all(torch.equal(a, b) for a, b in zip(have, want))


@pytest.mark.gpu
def test_errors_of_the_library_pass_through_both_ways(marshal, monkeypatch):
    dims = T.dims_of(T.V2, 4, torch.bfloat16)
    pool = torch.zeros(2, 64, 576, dtype=torch.bfloat16, device="cuda")
    cache = L.PagedCache(pool, T.i32([[0, 1]]), None)
    rows = torch.zeros(4, 576, dtype=torch.bfloat16, device="cuda")
    small = torch.zeros(4, dtype=torch.uint8, device="cuda")
    for m in (marshal, Declines):
        monkeypatch.setattr(L, "_marshal", m)
        with pytest.raises(L.MlaError):
            L.mla_cache_gather(dims, cache, T.i32([0, 4]), None, rows, small)
