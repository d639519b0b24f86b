"""A prompt through PromptLayer in one or several chunks, then decode steps on the same cache,
against the whole-sequence un-absorbed forward in 64 bits.

Tolerances are those of the decode step (bf16: max 2e-2, mean 5e-3 relative).  On
the way to an output about seven values in a row are rounded to bf16 (projection,
cache row, value, weight, head output, layer output, and the hidden state's products);
a rounding's root mean square is 2^-8 / (2 sqrt 3) times the value at most, so together
sqrt(7) 1.1e-3 = 3e-3.
"""

import dataclasses

import numpy as np
import pytest
import torch

import oracle
from mla_latent_kv_45_b200 import _lib as L
from mla_latent_kv_45_b200 import build, synth
from mla_latent_kv_45_b200.layer import DecodeLayer, PromptLayer
from mla_testlib import (assert_bf16_close, assert_fp32_close, dev, dev_weights, host, lib_dims,
                         oracle_dims)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    L.lib()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def offsets(lens):
    return [0] + list(np.cumsum(lens))


def run(wl, chunks, decode_steps=0, cache_format=L.MLA_CACHE_NATIVE):
    """chunks: per chunk the new tokens of each sequence.  Returns (outputs, hidden states) per
    sequence; decode steps follow where the sizes allow them."""
    B = len(chunks[0])
    W = synth.make_weights(wl)
    Wd = dev_weights(W, wl)
    dims = dataclasses.replace(lib_dims(wl), cache_format=cache_format)
    total = [sum(c[b] for c in chunks) + decode_steps for b in range(B)]
    hs = [synth.make_hidden(wl, tid=100 + b, n=max(total[b], 1))[:total[b]] for b in range(B)]
    ps = wl.page_size
    need = [-(-n // ps) for n in total]
    pages = sum(need) + 2
    table = np.full((B, max(need + [1])), -1, dtype=np.int32)
    order, at = np.random.RandomState(3).permutation(pages), 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    if cache_format == L.MLA_CACHE_INT8:
        pool = torch.zeros(pages, ps, 656, dtype=torch.uint8, device="cuda")
    else:
        pool = torch.zeros(pages, ps, wl.row, dtype=dims.torch_dtype, device="cuda")
    cache = L.PagedCache(pool, torch.from_numpy(table).cuda(), None)
    outs, done = [[] for _ in range(B)], [0] * B
    for c in chunks:
        h = np.concatenate([hs[b][done[b]:done[b] + c[b]] for b in range(B)])
        rows = [d + n for d, n in zip(done, c)]
        layer = PromptLayer(dims, Wd, B, sum(c), sum(rows))
        u = host(layer.step(cache, dev(h, wl), i32(offsets(c)), i32(done), i32(offsets(rows))))
        assert layer.device_error() == 0
        o = offsets(c)
        for b in range(B):
            outs[b].append(u[o[b]:o[b + 1]])
        done = rows
    for _ in range(decode_steps):
        layer = DecodeLayer(dims, Wd, B)
        cache.seq_lens = i32([d + 1 for d in done])
        h = np.stack([hs[b][done[b]] for b in range(B)])
        u = host(layer.step(cache, dev(h, wl), i32(done)))
        assert layer.device_error() == 0
        for b in range(B):
            outs[b].append(u[b:b + 1])
        done = [d + 1 for d in done]
    refs = [oracle.forward_naive(h, W, oracle_dims(wl)) if len(h) else h for h in hs]
    return [np.concatenate(o) for o in outs], refs


def test_fp32_prompts_in_chunks_then_decode():
    outs, refs = run(synth.TINY, [[20, 1, 0, 7], [13, 30, 5, 0]], decode_steps=3)
    for o, r in zip(outs, refs):
        assert_fp32_close(o, r, "u")


def test_bf16_prompt_then_decode():
    wl = synth.reduced(synth.V2_STEP128, "prompt", 91, 1, 0, 0, d_model=1024, d_q=512)
    outs, refs = run(wl, [[150, 33]], decode_steps=2)
    for o, r in zip(outs, refs):
        assert_bf16_close(o, r, "u")


def test_bf16_prompt_in_ragged_chunks():
    wl = synth.reduced(synth.V2_STEP128, "prompt", 92, 1, 0, 0, d_model=1024, d_q=512)
    outs, refs = run(wl, [[70, 1, 0], [45, 90, 3], [1, 0, 60]])
    for o, r in zip(outs, refs):
        assert_bf16_close(o, r, "u")


def test_int8_cache_prompt_is_consistent_with_decode():
    """Over 8-bit rows: the last token of a chunk and the same token decoded over the same
    cache agree (both read the quantised rows), within the tolerance of the decode step twice."""
    wl = synth.reduced(synth.V2_STEP128, "prompt", 93, 1, 0, 0, d_model=1024, d_q=512)
    W = synth.make_weights(wl)
    Wd = dev_weights(W, wl)
    dims = dataclasses.replace(lib_dims(wl), cache_format=L.MLA_CACHE_INT8)
    n = 130
    h = dev(synth.make_hidden(wl, n=n), wl)
    pool = torch.zeros(4, 64, 656, dtype=torch.uint8, device="cuda")
    cache = L.PagedCache(pool, i32([[2, 0, 3]]), i32([n]))
    layer = PromptLayer(dims, Wd, 1, n, n)
    u = layer.step(cache, h, i32([0, n]), None, i32([0, n]))
    assert layer.device_error() == 0
    dec = DecodeLayer(dims, Wd, 1)
    v = dec.step(cache, h[-1:].contiguous(), i32([n - 1]))
    assert dec.device_error() == 0
    g, r = host(u[-1:]), host(v)
    err = np.abs(g - r)
    assert err.max() <= 4e-2 and err.sum() / np.abs(r).sum() <= 1e-2


def test_captured_chunk_replays_with_other_lengths_and_on_another_stream():
    wl = synth.TINY
    W = synth.make_weights(wl)
    Wd = dev_weights(W, wl)
    dims = lib_dims(wl)
    hs = [synth.make_hidden(wl, tid=200 + b, n=40) for b in range(2)]
    pool = torch.zeros(8, 16, wl.row, device="cuda")
    cache = L.PagedCache(pool, i32([[0, 5, 2], [7, 1, 4]]), None)
    layer = PromptLayer(dims, Wd, 2, 24, 62)      # the last chunk leaves 35 + 27 rows
    h = torch.zeros(24, wl.d_model, device="cuda")
    cu, ctx, rows = i32([0, 12, 24]), i32([0, 0]), i32([0, 12, 24])
    h.copy_(dev(np.concatenate([hs[0][:12], hs[1][:12]]), wl))
    g = layer.capture(cache, h, cu, ctx, rows)
    refs = [oracle.forward_naive(x, W, oracle_dims(wl)) for x in hs]
    done = [0, 0]
    for new in ([12, 12], [20, 4], [3, 11]):
        o = offsets(new)
        h[:o[-1]] = dev(np.concatenate([hs[b][done[b]:done[b] + new[b]] for b in range(2)]), wl)
        cu.copy_(i32(o))
        ctx.copy_(i32(done))
        rows.copy_(i32(offsets([d + n for d, n in zip(done, new)])))
        out = host(g.replay())
        assert layer.device_error() == 0
        for b in range(2):
            assert_fp32_close(out[o[b]:o[b + 1]], refs[b][done[b]:done[b] + new[b]], f"seq {b}")
        done = [d + n for d, n in zip(done, new)]
    # a layer whose rows do not hold all of them says so
    small = PromptLayer(dims, Wd, 2, 24, 48)
    before = pool.clone()
    small.step(cache, h, cu, i32([d - n for d, n in zip(done, [3, 11])]), rows)
    assert small.device_error() == 6
    assert torch.equal(pool, before)      # (the same rows were appended again)
    # the same chunk on a stream of its own
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    want = layer.out.clone()
    ctx.copy_(i32([d - n for d, n in zip(done, [3, 11])]))
    torch.cuda.synchronize()
    got = layer.step(cache, h, cu, ctx, rows, side)
    side.synchronize()
    assert torch.equal(got[:14], want[:14])


def test_refuses_sizes_that_its_buffers_do_not_have():
    wl = synth.TINY
    dims, Wd = lib_dims(wl), dev_weights(synth.make_weights(wl), wl)
    for sizes in ((0, 4, 4), (1, 0, 4), (1, 4, 0)):
        with pytest.raises(ValueError):
            PromptLayer(dims, Wd, *sizes)
    layer = PromptLayer(dims, Wd, 1, 4, 4)
    cache = L.PagedCache(torch.zeros(1, 16, wl.row, device="cuda"), i32([[0]]), None)
    x = layer.x.data_ptr()
    for n in (3, 5):
        with pytest.raises(ValueError):
            layer.step(cache, torch.zeros(n, wl.d_model, device="cuda"), i32([0, n]), None,
                       i32([0, n]))
    assert layer.x.shape[0] == 4 and layer.x.data_ptr() == x
    layer.step(cache, torch.ones(4, wl.d_model, device="cuda"), i32([0, 4]), None, i32([0, 4]))
    assert layer.device_error() == 0
