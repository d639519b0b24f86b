"""Sequences beside bad ones, beside rows of no sequence and beside calls on other streams:
their own results, looked at row by row."""

import math

import pytest
import torch

from mla_latent_kv_45_b200 import _lib as L
from mla_latent_kv_45_b200 import build
from prompt_testlib import (TINY, V2, attn_inputs, attn_ref, check_attn, dims_of, i32, offsets,
                            run_attn, workspace)

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    L.lib()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


# offsets of the queries and keys, the bad sequence, heads, key heads, type
BAD = {
    "cut keys, queries past the end": ([3, 20, 101], [100, 2100, 4000], 1, 2, 2, BF),
    "cut keys, keys past the end": ([3, 20, 90], [100, 2100, 4101], 1, 2, 2, BF),
    "cut keys, first in front": ([-1, 20, 90], [100, 2100, 4000], 0, 2, 2, BF),
    "cut keys, grouped": ([3, 20, 90, 101], [0, 2100, 2500, 4000], 2, 16, 1, BF),
    "tiles": ([0, 40, 60, 101], [0, 40, 900, 1000], 2, 40, 40, BF),
    "few rows": ([0, 4, 20, 8, 30], [0, 50, 60, 90, 100], 2, 40, 40, BF),
    "fp32": ([0, 40, 60, 101], [0, 40, 90, 100], 2, 4, 2, F32),
}


@pytest.mark.parametrize("name", BAD)
def test_sequences_beside_a_bad_one(name):
    """A bad sequence's rows keep what they held; the others' are right, cut or not (a bad one
    changes how many pieces there are, so the bits of a cut call may differ).  Offsets that
    descend make the sequences on both sides overlap: a row that two of them have may hold the
    result of either and is not compared."""
    cu_q, cu_k, bad, heads, kv, dtype = BAD[name]
    dims = dims_of(V2 if dtype == BF else TINY, heads, dtype)
    n_q, n_k = 100, 4100
    t = attn_inputs(dims, n_q, n_k, kv, 43)
    ws = workspace(dims, len(cu_q) - 1, n_q)
    out = torch.full((n_q, heads, dims.d_v), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((n_q, heads), 7.0, device="cuda")
    L.mla_prompt_attn(dims, t["q_nope"], t["q_rope"], t["k_nope"], t["k_rope"], t["v"], i32(cu_q),
                      i32(cu_k), out, lse, ws)
    assert L.mla_get_device_error(ws) == 6
    owners = torch.zeros(n_q, dtype=torch.int32, device="cuda")
    for b in range(len(cu_q) - 1):
        if b != bad:
            owners[cu_q[b]:cu_q[b + 1]] += 1
    assert (out[owners == 0] == 7).all() and (lse[owners == 0] == 7).all()
    for b in range(len(cu_q) - 1):
        if b != bad:
            o, e = out.clone(), lse.clone()
            (rows, want, want_lse, _, _), = attn_ref(dims, t, cu_q[b:b + 2], cu_k[b:b + 2])
            two = owners[rows] > 1
            o[rows][two], e[rows][two] = want[two].to(dtype), want_lse[two].float()
            check_attn(dims, t, cu_q[b:b + 2], cu_k[b:b + 2], o, e, b)
    # the next call on this workspace, without the bad sequence
    good_q = cu_q[:bad] + [max(cu_q[bad], 0)] * (len(cu_q) - bad)
    good_k = cu_k[:bad] + [max(cu_k[bad], 0)] * (len(cu_k) - bad)
    out, lse = run_attn(dims, t, good_q, good_k, ws=ws)
    check_attn(dims, t, good_q, good_k, out, lse)


@pytest.mark.parametrize("dtype,n,k", [(BF, (70, 130), (100, 150)), (BF, (70, 130), (1500, 2000)),
                                       (BF, (3, 5), (40, 50)), (F32, (70, 130), (100, 150))])
def test_rows_of_no_sequence_change_no_bit(dtype, n, k):
    """The same results, bit for bit, with NaN and infinities around the sequences as with
    zeros there."""
    dims = dims_of(V2, 2, dtype)
    cu_q, cu_k = offsets(n, 5), offsets(k, 9)
    t = attn_inputs(dims, cu_q[-1] + 55, cu_k[-1] + 41, 2, 11)
    runs = []
    for front, back in ((0.0, 0.0), (math.nan, math.inf), (-math.inf, math.nan)):
        s = {name: v.clone() for name, v in t.items()}
        for name in ("q_nope", "q_rope"):
            s[name][:cu_q[0]], s[name][cu_q[-1]:] = front, back
        for name in ("k_nope", "k_rope", "v"):
            s[name][:cu_k[0]], s[name][cu_k[-1]:] = front, back
        runs.append(run_attn(dims, s, cu_q, cu_k))
    check_attn(dims, t, cu_q, cu_k, *runs[0])
    for out, lse in runs[1:]:
        assert torch.equal(out, runs[0][0]) and torch.equal(lse, runs[0][1])


@pytest.mark.parametrize("new,total", [([300, 17, 513, 128], [300, 17, 513, 128]), ([60], [6000]),
                                       ([1, 3] * 40, [90, 40] * 40)])
def test_every_call_on_two_streams_gives_the_same_bits(new, total):
    """Each call has output of its own, so that all of them are compared."""
    dims = dims_of(V2, 8, BF)
    cu_q, cu_k = offsets(new), offsets(total)
    t = attn_inputs(dims, cu_q[-1], cu_k[-1], 8, 19)
    want, want_lse = run_attn(dims, t, cu_q, cu_k)
    check_attn(dims, t, cu_q, cu_k, want, want_lse)
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [workspace(dims, len(new), cu_q[-1]) for _ in range(2)]
    got = [(torch.empty_like(want), torch.empty_like(want_lse)) for _ in range(24)]
    cq, ck = i32(cu_q), i32(cu_k)
    torch.cuda.synchronize()
    for i, (o, e) in enumerate(got):
        L.mla_prompt_attn(dims, t["q_nope"], t["q_rope"], t["k_nope"], t["k_rope"], t["v"], cq, ck,
                          o, e, spaces[i % 2], streams[i % 2])
    torch.cuda.synchronize()
    assert all(L.mla_get_device_error(ws) == 0 for ws in spaces)
    for o, e in got:
        assert torch.equal(o, want) and torch.equal(e, want_lse)
