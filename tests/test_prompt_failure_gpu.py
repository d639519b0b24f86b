"""Bounded waits of the prompt attention kernel: one that runs out is reported, and the workspace,
whose counters outlive a call, serves the next call as before.

No fault is made and nothing is withheld: mla_debug_prompt_timeout limits the waits to a few
microseconds, and the warps that write a block's output wait for all of its steps (1.2 us
each), so that a block over many keys runs into the limit.  What the kernel has in flight then it
waits for.
"""

import pytest
import torch

from mla_latent_kv_45_b200 import _lib as L
from mla_latent_kv_45_b200 import build
from prompt_testlib import V2, attn_inputs, check_attn, dims_of, i32, offsets, workspace

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    L.lib()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    yield
    L.mla_debug_prompt_timeout(False)


def test_the_hook_refuses_no_limit():
    with pytest.raises(L.MlaError) as e:
        L.mla_debug_prompt_timeout(True, 0)
    assert e.value.status == 1


# new tokens, keys, heads, key heads, whether the limits are sure to be reached
CASES = {
    "whole keys": ([6000], [6000], 4, 4, True),                    # 96 blocks of up to 75 steps
    "cut keys": ([200], [60000], 2, 2, True),                      # 148 pieces of 10 steps
    "ragged": ([700, 0, 333, 1, 90], [1411, 0, 5000, 900, 91], 16, 16, True),
    "grouped": ([300, 800], [2000, 3333], 64, 8, True),
    "no keys between": ([200, 30] * 20, [0, 3000] * 20, 4, 2, True),
    "many sequences": ([17 + i % 30 for i in range(700)], [60 + i % 50 for i in range(700)], 2, 1,
                       False),                                     # one or two steps each
}


@pytest.mark.parametrize("limit_us", [8, 4, 2, 1])
@pytest.mark.parametrize("name", CASES)
def test_wait_that_runs_out_is_reported_and_the_next_call_is_right(name, limit_us):
    new, total, heads, kv, sure = CASES[name]
    dims = dims_of(V2, heads, BF)
    cu_q, cu_k = offsets(new), offsets(total)
    t = attn_inputs(dims, cu_q[-1], cu_k[-1], kv, 3)
    ws = workspace(dims, len(new), cu_q[-1])
    out = torch.empty(cu_q[-1], heads, 128, dtype=BF, device="cuda")
    lse = torch.empty(cu_q[-1], heads, device="cuda")
    cq, ck = i32(cu_q), i32(cu_k)

    def call():
        L.mla_prompt_attn(dims, t["q_nope"], t["q_rope"], t["k_nope"], t["k_rope"], t["v"], cq, ck,
                          out, lse, ws)
        return L.mla_get_device_error(ws)

    assert call() == 0
    want, want_lse = out.clone(), lse.clone()
    for _ in range(3):
        L.mla_debug_prompt_timeout(True, limit_us)
        try:
            st = call()
        finally:
            L.mla_debug_prompt_timeout(False)
        assert st == 7 or not sure and st == 0            # MLA_ERR_TIMEOUT
        assert L.mla_get_device_error(ws) == 0            # reading clears it
        out.fill_(7)
        lse.fill_(7)
        assert call() == 0
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    check_attn(dims, t, cu_q, cu_k, out, lse)
