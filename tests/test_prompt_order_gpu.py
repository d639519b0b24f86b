"""The order of the attention kernel's asynchronous steps: cases whose results hang on a wait or
a fence and on nothing else."""

import pytest
import torch

from mla_latent_kv_45_b200 import _lib as L
from mla_latent_kv_45_b200 import build
from prompt_testlib import V2, attn_inputs, check_attn, dims_of, offsets, run_attn, workspace

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    L.lib()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("new,ctx,heads,kv", [([1500], [0], 8, 8), ([600, 900, 40], [200, 0, 700], 64, 64),
                                              ([300, 70], [500, 900], 64, 8)])
def test_maximum_that_never_moves(new, ctx, heads, kv):
    """The first key of a sequence outweighs the others a little, so no step rescales O: the
    weights of a step are stored over those that the product before has just read, in long
    items and at the first step of the items behind them, time after time."""
    dims = dims_of(V2, heads, BF)
    total = [a + b for a, b in zip(new, ctx)]
    cu_q, cu_k = offsets(new), offsets(total)
    t = attn_inputs(dims, cu_q[-1], cu_k[-1], kv, sum(new))
    t["q_nope"] = (t["q_nope"].float() * 0.25 + 0.25).to(BF)
    t["k_nope"] = (t["k_nope"].float() * 0.25).to(BF)
    t["k_rope"] = (t["k_rope"].float() * 0.25).to(BF)
    t["k_nope"][[k for k in cu_k[:-1]]] = 2.0     # a score of about 4.6, the others' within 1
    ws = workspace(dims, len(new), cu_q[-1])
    out, lse = run_attn(dims, t, cu_q, cu_k, ws=ws)
    check_attn(dims, t, cu_q, cu_k, out, lse)
    for _ in range(20):
        again, lse2 = run_attn(dims, t, cu_q, cu_k, ws=ws)
        assert torch.equal(again, out) and torch.equal(lse2, lse)
