"""Refusals of the prompt calls, on the host: no launch, so made-up addresses do."""

import ctypes

import pytest
import torch

from mla_latent_kv_45_b200 import _lib as L
from mla_latent_kv_45_b200 import build

A = 0x10000       # a 16-byte aligned address that nothing dereferences
OK, ARG, SHAPE, ALIGN, WS = 0, 1, 2, 3, 4
V2 = L.Dims(128, 512, 64, 128, 128, 64, L.MLA_BF16)
TINY = L.Dims(4, 16, 8, 8, 8, 16, L.MLA_FP32)
BIG = 1 << 30


@pytest.fixture(scope="module")
def lib():
    build.build()
    return L.lib()


def heads(ptr=A, token=128 * 64, head=64):
    return ctypes.byref(L._Heads(ptr, token, head))


def append(lib, dims=V2, cache=None, batch=2, n=10, x=A, xd=0, xs=576, gamma=A, cu=A, ctx=A, q="q",
           qo="q", ws=A, wsb=BIG):
    d = dims.c()
    c = L._Cache(A, 8, A, 4, None) if cache is None else cache
    q = heads() if q == "q" else q
    qo = heads() if qo == "q" else qo
    return lib.mla_prompt_append(ctypes.byref(d), ctypes.byref(c), batch, n, x, xd, xs, gamma,
                                 cu, ctx, q, qo, ws, wsb, None)


def gather(lib, dims=V2, cache=None, batch=2, n=10, cu=A, first=None, rows=A, ws=A, wsb=BIG):
    d = dims.c()
    c = L._Cache(A, 8, A, 4, None) if cache is None else cache
    return lib.mla_cache_gather(ctypes.byref(d), ctypes.byref(c), batch, n, cu, first, rows, ws,
                                wsb, None)


def attn(lib, dims=V2, batch=2, n_q=10, n_k=10, kv=128, qn=None, qr=None, kn=None, kr=A, krs=64,
         v=None, cu_q=A, cu_k=A, out=A, lse=A, ws=A, wsb=BIG):
    d = dims.c()
    wide = lambda h: heads(A, 128 * 128, 128) if h is None else h  # noqa: E731
    return lib.mla_prompt_attn(ctypes.byref(d), batch, n_q, n_k, kv, wide(qn),
                               heads() if qr is None else qr, wide(kn), kr, krs, wide(v), cu_q,
                               cu_k, out, lse, ws, wsb, None)


def test_workspace_size(lib):
    size = L.mla_prompt_workspace_size
    assert size(V2, 4, 0) > 0 and size(V2, 4, 100000) > size(V2, 4, 1000)
    sizes = [size(L.Dims(16, 512, 64, 128, 128, 64), b, n) for b, n in
             ((1, 1), (1, 100), (3, 100), (3, 3001), (70, 3001), (70, 90000))]
    assert sizes == sorted(sizes)
    assert size(V2, 0, 10) == 0 and size(V2, 1, -1) == 0
    assert size(L.Dims(257, 512, 64, 128, 128, 64), 1, 1) == 0
    assert size(L.Dims(16, 512, 64, 128, 128, 1), 1, 1) > 0
    assert size(L.Dims(16, 512, 64, 64, 128, 64), 1, 1) == 0
    assert size(L.Dims(4, 18, 8, 8, 8, 16, L.MLA_FP32), 1, 1) == 0


def test_append_refusals(lib):
    assert append(lib, L.Dims(0, 512, 64, 128, 128, 64)) == ARG
    assert append(lib, L.Dims(8, 256, 64, 128, 128, 64)) == SHAPE
    assert append(lib, L.Dims(8, 512, 64, 128, 128, 0)) == ARG
    assert append(lib, L.Dims(4, 16, 8, 8, 8, 16, L.MLA_FP32, cache_format=1)) == SHAPE
    for bad in (dict(x=None), dict(gamma=None), dict(cu=None), dict(batch=0), dict(n=-1),
                dict(xs=575), dict(xs=0), dict(xd=2), dict(xd=-1), dict(ws=None), dict(q=None), dict(qo=None),
                dict(q=heads(None)), dict(q=heads(A, 8192, 63)), dict(qo=heads(A, 63, 64)),
                dict(q=heads(A, 0, 64)), dict(qo=heads(A, 8192, -64)),
                dict(cache=L._Cache(None, 8, A, 4, None)), dict(cache=L._Cache(A, 0, A, 4, None)),
                dict(cache=L._Cache(A, 8, None, 4, None)), dict(cache=L._Cache(A, 8, A, 0, None))):
        assert append(lib, **bad) == ARG, bad
    for bad in (dict(x=A + 8), dict(xs=580), dict(gamma=A + 2), dict(cu=A + 2), dict(ctx=A + 1),
                dict(ws=A + 4), dict(q=heads(A + 8)), dict(qo=heads(A, 8196, 64)),
                dict(q=heads(A, 8192 + 64, 66)), dict(cache=L._Cache(A + 8, 8, A, 4, None))):
        assert append(lib, **bad) == ALIGN, bad
    assert append(lib, wsb=100) == WS
    assert append(lib, xd=1, wsb=100) == WS        # fp32 x beside bf16 rows
    assert append(lib, TINY, xd=0) == ARG
    assert append(lib, n=0) == OK                  # nothing to do: no launch


def test_gather_refusals(lib):
    for bad in (dict(cu=None), dict(rows=None), dict(batch=0), dict(n=-1), dict(ws=None)):
        assert gather(lib, **bad) == ARG, bad
    for bad in (dict(cu=A + 1), dict(first=A + 2), dict(rows=A + 8), dict(ws=A + 8)):
        assert gather(lib, **bad) == ALIGN, bad
    assert gather(lib, wsb=255) == WS
    assert gather(lib, n=0, rows=None) == OK


def test_attn_refusals(lib):
    assert attn(lib, L.Dims(128, 512, 64, 64, 128, 64)) == SHAPE
    assert attn(lib, L.Dims(300, 512, 64, 128, 128, 64)) == SHAPE
    assert attn(lib, L.Dims(128, 512, 64, 128, 128, 64, 5)) == ARG
    for bad in (dict(batch=0), dict(n_q=-1), dict(n_k=-1), dict(kv=0), dict(kv=3), dict(kv=256),
                dict(cu_q=None), dict(cu_k=None), dict(out=None), dict(kr=None), dict(ws=None),
                dict(qn=heads(None)), dict(kn=heads(A, 0, 128)), dict(v=heads(A, 16384, 127)),
                dict(qr=heads(A, 63, 64)), dict(krs=63), dict(krs=-64)):
        assert attn(lib, **bad) == ARG, bad
    for bad in (dict(cu_q=A + 2), dict(cu_k=A + 1), dict(out=A + 8), dict(lse=A + 2),
                dict(qn=heads(A + 8, 16384, 128)), dict(kr=A + 4), dict(krs=68), dict(ws=A + 8),
                dict(kn=heads(A, 16388, 128)), dict(v=heads(A, 16384, 132))):
        assert attn(lib, **bad) == ALIGN, bad
    assert attn(lib, wsb=L.mla_prompt_workspace_size(V2, 2, 10) - 1) == WS
    assert attn(lib, n_q=0, out=None) == OK


def test_python_refusals(lib):
    """The binding checks shapes, types and devices before it takes an address."""
    bf = dict(dtype=torch.bfloat16)
    d = L.Dims(2, 512, 64, 128, 128, 64, L.MLA_BF16)
    cu = torch.tensor([0, 3], dtype=torch.int32)
    ws = torch.zeros(1024, dtype=torch.uint8)
    good = dict(q_nope=torch.zeros(3, 2, 128, **bf), q_rope=torch.zeros(3, 2, 64, **bf),
                k_nope=torch.zeros(3, 1, 128, **bf), k_rope=torch.zeros(3, 64, **bf),
                v=torch.zeros(3, 1, 128, **bf), cu_q=cu, cu_k=cu,
                out=torch.zeros(3, 2, 128, **bf), lse=torch.zeros(3, 2))
    for bad in (dict(q_nope=torch.zeros(3, 2, 64, **bf)), dict(q_rope=torch.zeros(4, 2, 64, **bf)),
                dict(q_nope=torch.zeros(3, 2, 128)), dict(v=torch.zeros(3, 2, 128, **bf)),
                dict(k_rope=torch.zeros(3, 1, 64, **bf)), dict(cu_q=cu.long()),
                dict(cu_k=torch.zeros(3, dtype=torch.int32)), dict(out=torch.zeros(3, 256, **bf)),
                dict(lse=torch.zeros(2, 3)), dict(lse=torch.zeros(3, 2, **bf)),
                dict(out=torch.zeros(3, 128, 2, **bf).transpose(1, 2)),
                dict(k_nope=torch.zeros(3, 128, 1, **bf).transpose(1, 2)[:, :, ::1][..., :64]),
                dict()):      # the last: tensors of the host
        with pytest.raises(ValueError):
            L.mla_prompt_attn(d, **{**good, **bad}, ws=ws)
    cache = L.PagedCache(torch.zeros(2, 64, 576, **bf), torch.zeros(1, 2, dtype=torch.int32), None)
    app = dict(x=torch.zeros(3, 576, **bf), gamma=torch.ones(512, **bf), cu_tokens=cu,
               ctx_lens=torch.zeros(1, dtype=torch.int32))
    for bad in (dict(x=torch.zeros(3, 512, **bf)), dict(x=torch.zeros(576, 3, **bf).T),
                dict(gamma=torch.ones(512)), dict(ctx_lens=torch.zeros(2, dtype=torch.int32)),
                dict(q_rope=torch.zeros(3, 2, 64, **bf)), dict()):
        with pytest.raises(ValueError):
            L.mla_prompt_append(d, cache, **{**app, **bad}, ws=ws)
    int8 = L.Dims(2, 512, 64, 128, 128, 64, L.MLA_BF16, cache_format=L.MLA_CACHE_INT8)
    with pytest.raises(ValueError):
        L.mla_cache_gather(int8, cache, cu, None, torch.zeros(3, 576, **bf), ws)
    with pytest.raises(ValueError):
        L.mla_cache_gather(d, cache, cu, None, torch.zeros(3, 640, **bf), ws)
