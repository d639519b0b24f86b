"""Latent rows that are not finite, in a cache of 8-bit codes: the row reads back as NaN, as the
bf16 row would, instead of as zeros; the rows beside it are as they would be without it."""

import dataclasses
import math

import pytest
import torch

from mla_latent_kv_45_b200 import _lib as L
from mla_latent_kv_45_b200 import build
from prompt_testlib import V2, dims_of, i32, paged, row_values, rows_of, workspace

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    L.lib()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def bad_rows(x):
    """Rows 1, 3, 5 and 7 of x (16 rows) get one value each that is not finite."""
    x = x.clone()
    for r, c, v in ((1, 0, math.nan), (3, 511, math.inf), (5, 77, -math.inf), (7, 300, math.nan)):
        x[r, c] = v
    return x


ODD = [1, 3, 5, 7]
REST = [i for i in range(16) if i not in ODD]


@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_prompt_append_and_gather(dtype):
    dims = dims_of(V2, 2, BF, cache=L.MLA_CACHE_INT8)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(16, 576, generator=g, device="cuda").to(dtype)
    gamma = torch.ones(512, dtype=BF, device="cuda")
    ws = workspace(dims, 1, 16)
    cu = i32([0, 16])
    pools = []
    for v in (x, bad_rows(x)):
        cache = paged(dims, [16], 5)
        L.mla_prompt_append(dims, cache, v, gamma, cu, None, None, None, ws)
        rows = torch.empty(16, 576, dtype=BF, device="cuda")
        L.mla_cache_gather(dims, cache, cu, None, rows, ws)
        assert L.mla_get_device_error(ws) == 0
        raw = rows_of(cache, 0, 0, 16, 64)
        assert torch.equal(row_values(dims, raw)[REST], rows[REST].double())
        pools.append((raw, rows))
    (raw, rows), (raw2, rows2) = pools
    assert torch.equal(raw2[REST], raw[REST]) and torch.equal(rows2[REST], rows[REST])
    assert torch.isnan(rows2[ODD, :512]).all()
    assert torch.equal(rows2[:, 512:], rows[:, 512:])          # k_R is not quantised
    assert (raw2[ODD, :512] == 0).all() and (raw2[:, 644:] == 0).all()
    # a gamma that is not finite: every row
    gamma[9] = math.nan
    L.mla_prompt_append(dims, cache, x, gamma, cu, None, None, None, ws)
    L.mla_cache_gather(dims, cache, cu, None, rows, ws)
    assert torch.isnan(rows[:, :512]).all()


def test_decode_append_and_attention():
    """The append of a decode step does the same, and attention over such a row is NaN, that of
    the other sequences as before."""
    dims = dims_of(V2, 128, BF, cache=L.MLA_CACHE_INT8)
    native = dataclasses.replace(dims, cache_format=L.MLA_CACHE_NATIVE)
    g = torch.Generator(device="cuda").manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)  # noqa: E731
    batch, width = 16, 128
    h, w_dkv, w_kr, gamma = r(batch, width), r(512, width), r(64, width), torch.ones(512, dtype=BF, device="cuda")
    q_lat = r(batch, 128, 576)
    size = L.mla_workspace_size(dims, batch, width, 0, 0)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    L.mla_workspace_init(ws)
    pos = i32([0, 1, 2, 60, 0, 0, 63, 10] + [5] * 8)
    lens = (pos + 1).tolist()
    res = {}
    for name, d in (("int8", dims), ("native", native)):
        for what in ("good", "bad"):
            cache = paged(d, lens, 7)
            cache.seq_lens = pos + 1
            v = h.clone()
            if what == "bad":
                v[ODD, 3] = math.nan
            L.mla_cache_append(d, cache, v, w_dkv, w_kr, gamma, pos, ws)
            z = torch.empty(batch, 128, 512, dtype=BF, device="cuda")
            L.mla_decode_attn(d, cache, q_lat, z, None, 0, ws)
            assert L.mla_get_device_error(ws) == 0
            rows = torch.stack([row_values(d, rows_of(cache, b, int(pos[b]), 1, 64))[0]
                                for b in range(batch)])
            res[name, what] = rows, z
    for name in ("int8", "native"):
        (rows, z), (rows2, z2) = res[name, "good"], res[name, "bad"]
        assert torch.isfinite(rows).all() and torch.isfinite(z).all()
        assert torch.isnan(rows2[ODD]).all() and torch.isnan(z2[ODD]).all(), name
        assert torch.equal(rows2[REST], rows[REST]) and torch.equal(z2[REST], z[REST]), name
