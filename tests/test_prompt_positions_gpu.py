"""Positions at and outside the borders: what the append writes, rotates and leaves."""

import pytest
import torch

from mla_latent_kv_45_b200 import _lib as L
from mla_latent_kv_45_b200 import build
from prompt_testlib import (TINY, V2, close_rotated, dims_of, i32, paged, rotate_ref, workspace)

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    L.lib()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("layout", [L.MLA_ROPE_HALF, L.MLA_ROPE_INTERLEAVED])
@pytest.mark.parametrize("kind", ["bf16", "int8", "fp32"])
@pytest.mark.parametrize("ctx", [-3, -100, 2 ** 31 - 5, 2 ** 31 - 1, 1 << 20])
def test_queries_of_positions_without_a_page(kind, layout, ctx):
    """Rows of the second sequence, whose positions start at ctx, have no page (or, from -3 on,
    some have): queries at positions in [0, 2^31) are rotated, the others' output is left."""
    dtype = F32 if kind == "fp32" else BF
    dims = dims_of(TINY if kind == "fp32" else V2, 3, dtype, 16, layout,
                   L.MLA_CACHE_INT8 if kind == "int8" else L.MLA_CACHE_NATIVE)
    cache = paged(dims, [20, 20], 3)
    before = cache.pool.clone()
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(30, dims.d_c + dims.d_rope, generator=g, device="cuda").to(dtype)
    q = torch.randn(30, 3, dims.d_rope, generator=g, device="cuda").to(dtype)
    gamma = torch.ones(dims.d_c, dtype=dtype, device="cuda")
    out = torch.full_like(q, 7.0)
    ws = workspace(dims, 2, 30)
    L.mla_prompt_append(dims, cache, x, gamma, i32([0, 20, 30]), i32([0, ctx]), q, out, ws)
    assert L.mla_get_device_error(ws) == 6
    pos = torch.cat([torch.arange(20), torch.arange(10) + ctx]).cuda()      # 64 bits
    inside = (pos >= 0) & (pos < 2 ** 31)
    assert bool(inside[20:].any()) == (ctx != -100)
    ref, size = rotate_ref(q[inside], pos[inside], layout)
    assert close_rotated(out[inside], ref, size, dtype)
    assert (out[~inside] == 7).all()
    # rows were written at the first sequence's places and at the second's that exist
    used = torch.zeros(cache.pool.shape[:2], dtype=torch.bool, device="cuda")
    for b, at in ((0, pos[:20]), (1, pos[20:][(pos[20:] >= 0) & (pos[20:] < 20)])):
        used[cache.block_table[b].long()[at // 16], at % 16] = True
    assert torch.equal(cache.pool[~used].view(torch.uint8), before[~used].view(torch.uint8))
    for b in range(2):
        n = 20 if b == 0 else int(((pos[20:] >= 0) & (pos[20:] < 20)).sum())
        rows = cache.pool[cache.block_table[b].long()[0], :min(n, 16)]
        assert not torch.equal(rows, before[cache.block_table[b].long()[0], :min(n, 16)]) or n == 0
