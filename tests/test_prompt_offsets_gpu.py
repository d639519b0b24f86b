"""Offsets that do not ascend or that leave the packed rows: every call records them, wherever they
stand, and records nothing otherwise."""

import pytest
import torch

from mla_latent_kv_45_b200 import _lib as L
from mla_latent_kv_45_b200 import build
from prompt_testlib import TINY, V2, attn_inputs, dims_of, i32, offsets, workspace

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    L.lib()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


GOOD = [[0, 100], [0, 40, 100], [7, 7, 50, 50, 93], offsets([1] * 100), offsets([0] * 400 + [100] + [0] * 900),
        offsets([1, 0] * 100)]
BAD = [[0, 101], [0, 40, 130], [-5, 100], [-5, 0, 100], [0, 50, 40, 40], [0, 50, 20, 100], [0, 200, 100],
       [30, 20, 10], [2 ** 30, 2 ** 31 - 1], [-2 ** 31, 0], offsets([1] * 100)[:60] + [5] + [100] * 39,
       offsets([0] * 1300 + [101]), [3] * 700 + [2] + [3] * 700 + [100]]


def calls(kind, cu):
    """The status of each call with 100 packed rows."""
    dtype = F32 if kind == "fp32" else BF
    batch = len(cu) - 1
    dims = dims_of(TINY if kind == "fp32" else V2, 2, dtype, 64, L.MLA_ROPE_HALF,
                   L.MLA_CACHE_INT8 if kind == "int8" else L.MLA_CACHE_NATIVE)
    g = torch.Generator(device="cuda").manual_seed(4)
    width = dims.d_c + dims.d_rope
    if kind == "int8":
        pool = torch.zeros(2 * batch, 64, 656, dtype=torch.uint8, device="cuda")
    else:
        pool = torch.zeros(2 * batch, 64, width, dtype=dtype, device="cuda")
    table = torch.arange(2 * batch, dtype=torch.int32, device="cuda").view(batch, 2)
    cache = L.PagedCache(pool, table, None)
    x = torch.randn(100, width, generator=g, device="cuda").to(dtype)
    gamma = torch.ones(dims.d_c, dtype=dtype, device="cuda")
    rows = torch.zeros(100, width, dtype=dtype, device="cuda")
    q = torch.randn(100, 2, dims.d_rope, generator=g, device="cuda").to(dtype)
    t = attn_inputs(dims, 100, 100, 2, 5)
    out = torch.zeros(100, 2, dims.d_v, dtype=dtype, device="cuda")
    whole = torch.full((L.mla_prompt_workspace_size(dims, batch, 100) + 4096,), 7, dtype=torch.uint8,
                       device="cuda")
    ws = whole[:-4096]
    L.mla_workspace_init(ws)
    cud, st = i32(cu), []
    L.mla_prompt_append(dims, cache, x, gamma, cud, None, None, None, ws)
    st.append(L.mla_get_device_error(ws))
    L.mla_prompt_append(dims, cache, x, gamma, cud, None, q, q, ws)
    st.append(L.mla_get_device_error(ws))
    L.mla_cache_gather(dims, cache, cud, None, rows, ws)
    st.append(L.mla_get_device_error(ws))
    if kind != "int8":
        L.mla_prompt_attn(dims, t["q_nope"], t["q_rope"], t["k_nope"], t["k_rope"], t["v"], cud, cud,
                          out, None, ws)
        st.append(L.mla_get_device_error(ws))
    assert (whole[-4096:] == 7).all()
    return st


@pytest.mark.parametrize("kind", ["bf16", "int8", "fp32"])
def test_good_offsets_record_nothing(kind):
    for cu in GOOD:
        assert set(calls(kind, cu)) == {0}, cu[:6]


@pytest.mark.parametrize("kind", ["bf16", "int8", "fp32"])
def test_bad_offsets_are_recorded(kind):
    for cu in BAD:
        assert set(calls(kind, cu)) == {6}, cu[:6]
