"""Cache append of packed rows and cache gather against their definitions in 64 bits."""

import pytest
import torch

import oracle
from mla_latent_kv_45_b200 import _lib as L
from mla_latent_kv_45_b200 import build
from prompt_testlib import (TINY, V2, close_normed, close_rotated, dims_of, i32, norm_ref, offsets,
                            paged, rotate_ref, row_values, rows_of, workspace)

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
HALF, INTER = L.MLA_ROPE_HALF, L.MLA_ROPE_INTERLEAVED


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    L.lib()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def inputs(dims, n, seed, scale=1.4):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = dims.torch_dtype
    x = (scale * torch.randn(n, dims.d_c + dims.d_rope, generator=g, device="cuda")).to(t)
    gamma = (1 + 0.1 * torch.randn(dims.d_c, generator=g, device="cuda")).to(t)
    q = torch.randn(n, dims.n_heads, dims.d_rope, generator=g, device="cuda").to(t)
    return x, gamma, q


def check_rows(dims, cache, before, new, ctx, x, gamma, cu):
    """The written slots hold the rows, every other byte of the pool is as it was."""
    page, t = dims.page_size, dims.torch_dtype
    touched = torch.zeros(cache.pool.shape[:2], dtype=torch.bool, device="cuda")
    for b, n in enumerate(new):
        pos = torch.arange(ctx[b], ctx[b] + n, device="cuda")
        touched[cache.block_table[b].long()[pos // page], pos % page] = True
        raw = rows_of(cache, b, ctx[b], n, page)
        xs = x[cu[b]:cu[b + 1]]
        c = norm_ref(xs[:, :dims.d_c], gamma)
        k, size = rotate_ref(xs[:, dims.d_c:], pos, dims.rope_layout)
        vals = row_values(dims, raw)
        assert close_rotated(vals[:, dims.d_c:], k, size, t), b
        if dims.cache_format == L.MLA_CACHE_INT8:
            q, e = oracle.quantize_int8_pow2(c.cpu().numpy())
            want = torch.from_numpy(oracle.dequantize_int8_pow2(q, e)).cuda()
            assert torch.equal(vals[:, :512], want), b
            assert (raw[:, 644:] == 0).all(), b
        else:
            assert close_normed(vals[:, :dims.d_c], c, dims.d_c, t), b
    assert torch.equal(cache.pool[~touched].view(torch.uint8), before[~touched].view(torch.uint8))


CASES = [
    # new tokens, cached rows
    ([1], [0]),
    ([115], [0]),
    ([0, 64, 1, 65, 0], [5, 64, 63, 1, 0]),
    ([3, 200, 0, 31], [1000, 61, 7, 131041]),
]


@pytest.mark.parametrize("new,ctx", CASES)
@pytest.mark.parametrize("layout", [INTER, HALF])
@pytest.mark.parametrize("kind", ["bf16", "int8", "fp32"])
def test_append(new, ctx, layout, kind):
    dtype = F32 if kind == "fp32" else BF
    dims = dims_of(TINY if kind == "fp32" else V2, 5, dtype, 16 if kind == "fp32" else 64, layout,
                   L.MLA_CACHE_INT8 if kind == "int8" else L.MLA_CACHE_NATIVE)
    cu = offsets(new)
    cache = paged(dims, [a + b for a, b in zip(new, ctx)], 3, extra_pages=1)
    before = cache.pool.clone()
    x, gamma, q = inputs(dims, cu[-1], 5)
    out = torch.full_like(q, 7.0)
    ws = workspace(dims, len(new), cu[-1])
    L.mla_prompt_append(dims, cache, x, gamma, i32(cu), i32(ctx), q, out, ws)
    assert L.mla_get_device_error(ws) == 0
    check_rows(dims, cache, before, new, ctx, x, gamma, cu)
    pos = torch.cat([torch.arange(c, c + n, device="cuda") for n, c in zip(new, ctx)])
    ref, size = rotate_ref(q, pos, layout)
    assert close_rotated(out, ref, size, dtype)


@pytest.mark.parametrize("heads", [1, 3, 15, 16, 17, 127, 128, 129, 256])
def test_append_rotates_any_number_of_heads_in_place_and_in_slices(heads):
    dims = dims_of(V2, heads, BF)
    n = 37
    cache = paged(dims, [n + 10], 3)
    x, gamma, q = inputs(dims, n, heads)
    ws = workspace(dims, 1, n)
    pos = torch.arange(10, 10 + n, device="cuda")
    ref, size = rotate_ref(q, pos, INTER)
    wide = torch.full((n, heads, 192), 7.0, dtype=BF, device="cuda")
    L.mla_prompt_append(dims, cache, x, gamma, i32([0, n]), i32([10]), q, wide[..., 128:], ws)
    assert close_rotated(wide[..., 128:], ref, size, BF)
    assert (wide[..., :128] == 7).all()
    got = q.clone()
    L.mla_prompt_append(dims, cache, x, gamma, i32([0, n]), i32([10]), got, got, ws)
    assert torch.equal(got, wide[..., 128:])


@pytest.mark.parametrize("page", [1, 7, 64, 100])
def test_append_and_gather_with_other_pages_and_wide_rows(page):
    """Any page size, x as a slice of a wider product, no queries, no cached rows."""
    dims = dims_of(V2, 2, BF, page)
    new = [33, 0, 130]
    cu = offsets(new)
    cache = paged(dims, new, 7)
    before = cache.pool.clone()
    x, gamma, _ = inputs(dims, cu[-1], 9)
    wide = torch.zeros(cu[-1], 1024, dtype=BF, device="cuda")
    wide[:, 8:584] = x
    ws = workspace(dims, 3, cu[-1])
    L.mla_prompt_append(dims, cache, wide[:, 8:584], gamma, i32(cu), None, None, None, ws)
    assert L.mla_get_device_error(ws) == 0
    check_rows(dims, cache, before, new, [0, 0, 0], x, gamma, cu)
    rows = torch.empty(cu[-1], 576, dtype=BF, device="cuda")
    L.mla_cache_gather(dims, cache, i32(cu), None, rows, ws)
    assert L.mla_get_device_error(ws) == 0
    want = torch.cat([rows_of(cache, b, 0, n, page) for b, n in enumerate(new)])
    assert torch.equal(rows, want)


@pytest.mark.parametrize("kind", ["bf16", "int8"])
@pytest.mark.parametrize("layout", [INTER, HALF])
def test_append_of_fp32_projections(kind, layout):
    """Products left in fp32: normalised and rotated before the one rounding."""
    dims = dims_of(V2, 3, BF, 64, layout,
                   L.MLA_CACHE_INT8 if kind == "int8" else L.MLA_CACHE_NATIVE)
    new, ctx = [70, 0, 3], [5, 1, 200]
    cu = offsets(new)
    cache = paged(dims, [a + b for a, b in zip(new, ctx)], 33)
    before = cache.pool.clone()
    _, gamma, q = inputs(dims, cu[-1], 35)
    g = torch.Generator(device="cuda").manual_seed(36)
    wide = 1.4 * torch.randn(cu[-1], 600, generator=g, device="cuda")
    x = wide[:, 16:592]
    ws = workspace(dims, 3, cu[-1])
    L.mla_prompt_append(dims, cache, x, gamma, i32(cu), i32(ctx), q, q, ws)
    assert L.mla_get_device_error(ws) == 0
    check_rows(dims, cache, before, new, ctx, x, gamma, cu)


def test_append_of_zero_and_of_large_rows():
    """A row of zeros stays zero (code scale 1); values up to 1e30 normalise."""
    for fmt in (L.MLA_CACHE_NATIVE, L.MLA_CACHE_INT8):
        dims = dims_of(V2, 1, BF, cache=fmt)
        cache = paged(dims, [3], 3)
        before = cache.pool.clone()
        x, gamma, _ = inputs(dims, 3, 11)
        x[0] = 0
        x[1] *= 2.0 ** 50
        x[2] *= 2.0 ** -40
        ws = workspace(dims, 1, 3)
        L.mla_prompt_append(dims, cache, x, gamma, i32([0, 3]), None, None, None, ws)
        check_rows(dims, cache, before, [3], [0], x, gamma, [0, 3])


@pytest.mark.parametrize("kind", ["bf16", "int8", "fp32"])
def test_append_rows_outside_the_sequences_and_bad_places(kind):
    dtype = F32 if kind == "fp32" else BF
    dims = dims_of(TINY if kind == "fp32" else V2, 3, dtype, 16, INTER,
                   L.MLA_CACHE_INT8 if kind == "int8" else L.MLA_CACHE_NATIVE)
    cache = paged(dims, [40, 20], 3)
    cache.block_table[0, 1] = cache.pool.shape[0]      # page out of range for rows 16..31
    before = cache.pool.clone()
    x, gamma, q = inputs(dims, 70, 13)
    out = torch.full_like(q, 7.0)
    ws = workspace(dims, 2, 70)
    L.mla_prompt_append(dims, cache, x, gamma, i32([4, 44, 64]), None, q, out, ws)
    assert L.mla_get_device_error(ws) == 6
    assert L.mla_get_device_error(ws) == 0
    assert (out[:4] == 7).all() and (out[64:] == 7).all()
    pos = torch.cat([torch.arange(40), torch.arange(20)]).cuda()
    ref, size = rotate_ref(q[4:64], pos, INTER)
    assert close_rotated(out[4:64], ref, size, dtype)
    ok = torch.ones(40, dtype=torch.bool)
    ok[16:32] = False
    vals = row_values(dims, rows_of(cache, 1, 0, 20, 16))
    k, size = rotate_ref(x[44:64, dims.d_c:], torch.arange(20).cuda(), INTER)
    assert close_rotated(vals[:, dims.d_c:], k, size, dtype)
    used = torch.zeros(cache.pool.shape[:2], dtype=torch.bool, device="cuda")
    for b, rows in ((0, torch.arange(40)[ok]), (1, torch.arange(20))):
        rows = rows.cuda()
        used[cache.block_table[b].long()[rows // 16], rows % 16] = True
    assert torch.equal(cache.pool[~used].view(torch.uint8), before[~used].view(torch.uint8))
    # positions that no page covers, and a negative one
    for ctx in ([1 << 20, 0], [-100, 0], [2 ** 31 - 1, 0]):
        cache.pool.copy_(before)
        L.mla_prompt_append(dims, cache, x, gamma, i32([0, 40, 60]), i32(ctx), q, out, ws)
        assert L.mla_get_device_error(ws) == 6
        page0 = cache.block_table[0, 0].long()
        assert torch.equal(cache.pool[page0].view(torch.uint8), before[page0].view(torch.uint8))


@pytest.mark.parametrize("kind", ["bf16", "int8", "fp32"])
def test_gather(kind):
    dtype = F32 if kind == "fp32" else BF
    dims = dims_of(TINY if kind == "fp32" else V2, 3, dtype, 16 if kind == "fp32" else 64, INTER,
                   L.MLA_CACHE_INT8 if kind == "int8" else L.MLA_CACHE_NATIVE)
    page = dims.page_size
    lens, first = [1, 0, 200, 64, 65, 130], [0, 3, 17, 64, 63, 0]
    cache = paged(dims, [a + b for a, b in zip(lens, first)], 21)
    cu = offsets(lens, 2)
    rows = torch.full((cu[-1] + 5, dims.d_c + dims.d_rope), 7.0, dtype=dtype, device="cuda")
    ws = workspace(dims, len(lens), 1)
    L.mla_cache_gather(dims, cache, i32(cu), i32(first), rows, ws)
    assert L.mla_get_device_error(ws) == 0
    for b, n in enumerate(lens):
        want = row_values(dims, rows_of(cache, b, first[b], n, page))
        assert torch.equal(rows[cu[b]:cu[b + 1]].double(), want), b
    assert (rows[:2] == 7).all() and (rows[cu[-1]:] == 7).all()
    # a page outside the pool, and rows past the table: zeroed, recorded, the others read
    cache.block_table[2, 1] = -7
    L.mla_cache_gather(dims, cache, i32(cu), i32(first), rows, ws)
    assert L.mla_get_device_error(ws) == 6
    got = rows[cu[2]:cu[3]].double()
    pos = torch.arange(17, 217, device="cuda")
    bad = pos // page == 1
    assert (got[bad] == 0).all()
    want = row_values(dims, cache.pool[cache.block_table[2].long()[pos // page].clamp(min=0), pos % page])
    assert torch.equal(got[~bad], want[~bad])


def test_gather_many_short_sequences():
    dims = dims_of(V2, 1, BF)
    lens = [(5 * i) % 9 for i in range(1500)]
    cache = paged(dims, lens, 23)
    cu = offsets(lens)
    rows = torch.empty(cu[-1], 576, dtype=BF, device="cuda")
    ws = workspace(dims, len(lens), 1)
    L.mla_cache_gather(dims, cache, i32(cu), None, rows, ws)
    assert L.mla_get_device_error(ws) == 0
    want = torch.cat([rows_of(cache, b, 0, n, 64) for b, n in enumerate(lens) if n])
    assert torch.equal(rows, want)


def test_offsets_past_32_bits():
    """A pool of more than 2^31 values (4.9 GB): slots beyond it are written and read."""
    dims = dims_of(V2, 1, BF)
    num = 66000
    pool = torch.zeros(num, 64, 576, dtype=BF, device="cuda")
    table = i32([[num - 1, 3, num - 2]])
    cache = L.PagedCache(pool, table, None)
    x, gamma, _ = inputs(dims, 150, 25)
    ws = workspace(dims, 1, 150)
    L.mla_prompt_append(dims, cache, x, gamma, i32([0, 150]), None, None, None, ws)
    rows = torch.empty(150, 576, dtype=BF, device="cuda")
    L.mla_cache_gather(dims, cache, i32([0, 150]), None, rows, ws)
    assert L.mla_get_device_error(ws) == 0
    assert torch.equal(rows, rows_of(cache, 0, 0, 150, 64))
    assert close_normed(rows[:, :512], norm_ref(x[:, :512], gamma), 512, BF)
    assert (pool[4:8] == 0).all()


def test_offsets_that_descend_are_recorded():
    dims = dims_of(V2, 1, BF)
    cache = paged(dims, [64, 64, 64], 27)
    x, gamma, _ = inputs(dims, 100, 27)
    ws = workspace(dims, 3, 100)
    L.mla_prompt_append(dims, cache, x, gamma, i32([0, 50, 20, 100]), None, None, None, ws)
    assert L.mla_get_device_error(ws) == 6     # tokens 20..49 belong to no sequence
    rows = torch.full((100, 576), 7.0, dtype=BF, device="cuda")
    L.mla_cache_gather(dims, cache, i32([0, 50, 20, 100]), None, rows, ws)
    assert L.mla_get_device_error(ws) == 6


def test_captured_append_and_gather_read_their_offsets_at_replay():
    dims = dims_of(V2, 4, BF)
    cache = paged(dims, [300, 300], 29)
    x, gamma, q = inputs(dims, 120, 31)
    cu, ctx, call = i32([0, 60, 120]), i32([0, 0]), i32([0, 60, 120])
    out = torch.empty_like(q)
    rows = torch.full((400, 576), 7.0, dtype=BF, device="cuda")
    ws = workspace(dims, 2, 120)

    def both():
        L.mla_prompt_append(dims, cache, x, gamma, cu, ctx, q, out, ws)
        L.mla_cache_gather(dims, cache, call, None, rows, ws)

    both()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
    for new, old in (([60, 60], [0, 0]), ([100, 7], [60, 60]), ([0, 50], [160, 67])):
        total = [a + b for a, b in zip(new, old)]
        cu.copy_(i32(offsets(new)))
        ctx.copy_(i32(old))
        call.copy_(i32(offsets(total)))
        before = cache.pool.clone()
        g.replay()
        torch.cuda.synchronize()
        assert L.mla_get_device_error(ws) == 0
        check_rows(dims, cache, before, new, old, x, gamma, offsets(new))
        want = torch.cat([rows_of(cache, b, 0, n, 64) for b, n in enumerate(total)])
        assert torch.equal(rows[:sum(total)], want)
