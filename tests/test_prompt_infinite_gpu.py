"""Scores of -inf that a row sees: they weigh nothing beside others, and where a row sees no
others the formula gives 0 / 0 = NaN and lse = log 0 = -inf, in every kernel alike."""

import math

import pytest
import torch

from mla_latent_kv_45_b200 import _lib as L
from mla_latent_kv_45_b200 import build
from prompt_testlib import TINY, V2, attn_inputs, check_attn, dims_of, offsets, run_attn

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    L.lib()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


# new tokens, keys, heads, key heads, type, size
CASES = {
    "tiles": ([200, 0, 130, 40], [200, 30, 300, 17], 4, 4, BF, V2),
    "tiles, grouped": ([60, 33, 9], [60, 200, 4], 16, 2, BF, V2),
    "tiles, many sequences": ([40] * 600, [50] * 600, 1, 1, BF, V2),
    "cut keys": ([60], [3000], 3, 3, BF, V2),
    "cut keys, grouped, some see none": ([40, 90], [1700, 30], 8, 1, BF, V2),
    "few rows": ([3, 16, 1, 5], [200, 16, 40, 2], 2, 2, BF, V2),
    "few rows, many sequences": ([2, 5] * 90, [30, 4] * 90, 4, 2, BF, V2),
    "fp32": ([33, 0, 7, 40], [50, 4, 7, 11], 4, 2, F32, TINY),
}


def minus_infinity(t, dims, keys):
    """The given keys score -inf: the queries' first value is 1, the keys' is -inf."""
    t["q_nope"][..., 0] = 1
    t["k_nope"][..., 0] = 0
    t["k_nope"][keys, :, 0] = -math.inf


@pytest.mark.parametrize("name", CASES)
def test_every_key_of_a_sequence_scores_minus_infinity(name):
    new, total, heads, kv, dtype, size = CASES[name]
    dims = dims_of(size, heads, dtype)
    cu_q, cu_k = offsets(new), offsets(total)
    t = attn_inputs(dims, cu_q[-1], cu_k[-1], kv, 5)
    minus_infinity(t, dims, slice(0, 0))
    want, want_lse = run_attn(dims, t, cu_q, cu_k)
    check_attn(dims, t, cu_q, cu_k, want, want_lse)
    for bad in range(0, len(new), max(1, len(new) // 4)):
        minus_infinity(t, dims, slice(cu_k[bad], cu_k[bad + 1]))
        out, lse = run_attn(dims, t, cu_q, cu_k)
        see = torch.arange(new[bad], device="cuda") + total[bad] - new[bad] + 1
        mine, mine_lse = out[cu_q[bad]:cu_q[bad + 1]], lse[cu_q[bad]:cu_q[bad + 1]]
        assert torch.isneginf(mine_lse).all(), bad
        assert torch.isnan(mine[see > 0]).all(), bad
        assert (mine[see <= 0] == 0).all(), bad
        # the other sequences are as before
        mine.copy_(want[cu_q[bad]:cu_q[bad + 1]])
        mine_lse.copy_(want_lse[cu_q[bad]:cu_q[bad + 1]])
        assert torch.equal(out, want) and torch.equal(lse, want_lse), bad


@pytest.mark.parametrize("name", CASES)
def test_some_keys_score_minus_infinity(name):
    """Every key but the last and every seventh: a row has its first finite score early, late or
    in a piece of the keys of its own; rows before the first one get NaN and -inf."""
    new, total, heads, kv, dtype, size = CASES[name]
    dims = dims_of(size, heads, dtype)
    cu_q, cu_k = offsets(new), offsets(total)
    t = attn_inputs(dims, cu_q[-1], cu_k[-1], kv, 6)
    bad = torch.ones(cu_k[-1], dtype=torch.bool, device="cuda")
    first = []
    for b, m in enumerate(total):
        bad[cu_k[b] + m // 2:cu_k[b + 1]:7] = False
        first.append(m // 2)
        if m:
            bad[cu_k[b + 1] - 1] = False
    minus_infinity(t, dims, bad)
    out, lse = run_attn(dims, t, cu_q, cu_k)
    for b, n in enumerate(new):
        see = torch.arange(n, device="cuda") + total[b] - n + 1
        none = (see > 0) & (see <= first[b])
        rows = slice(cu_q[b], cu_q[b + 1])
        assert torch.isnan(out[rows][none]).all() and torch.isneginf(lse[rows][none]).all(), b
        out[rows][none], lse[rows][none] = 0, -math.inf
    # the others against the formula over the keys that are left: -inf times a query's 1 is the
    # only infinite product, so the scores that count do not change when it is taken out
    s = dict(t, k_nope=t["k_nope"].clone())
    s["k_nope"][..., 0] = 0
    check_without(dims, s, cu_q, cu_k, out, lse, bad)


def check_without(dims, t, cu_q, cu_k, out, lse, bad):
    """Bounds as in check_attn, over the keys that are not `bad`."""
    d = dims.d_nope + dims.d_rope
    bf = dims.torch_dtype == BF
    rep = dims.n_heads // t["k_nope"].shape[1]
    for b in range(len(cu_q) - 1):
        q0, q1, k0, k1 = cu_q[b], cu_q[b + 1], cu_k[b], cu_k[b + 1]
        n, m = q1 - q0, k1 - k0
        if n == 0 or m == 0:
            continue
        q = torch.cat([t["q_nope"][q0:q1], t["q_rope"][q0:q1]], -1).double().transpose(0, 1)
        kr = t["k_rope"][k0:k1, None].expand(-1, t["k_nope"].shape[1], -1)
        k = torch.cat([t["k_nope"][k0:k1], kr], -1).double().transpose(0, 1)
        k = k.repeat_interleave(rep, 0)
        v = t["v"][k0:k1].double().transpose(0, 1).repeat_interleave(rep, 0)
        seen = (torch.arange(m, device="cuda")[None]
                <= torch.arange(n, device="cuda")[:, None] + m - n) & ~bad[k0:k1]
        x = ((q @ k.transpose(1, 2)) / math.sqrt(d)).masked_fill(~seen, -math.inf)
        size = ((q.abs() @ k.abs().transpose(1, 2)) / math.sqrt(d)).masked_fill(~seen, 0.0)
        e = torch.logsumexp(x, -1)
        some = torch.isfinite(e)
        p = torch.exp(x - e[..., None]).masked_fill(~seen, 0.0).nan_to_num(0.0)
        o, a, big = p @ v, p @ v.abs(), size.amax(-1)
        ds = d * 2.0 ** -23 * big + (2.0 ** -17 if bf else 2.0 ** -21)
        tol = 2 * ds[..., None] * a + 2.0 ** -24 * (m + 8) * a
        if bf:
            tol = tol + 2.0 ** -8 * (a + o.abs())
        got, ge = out[q0:q1].double().transpose(0, 1), lse[q0:q1].double().transpose(0, 1)
        assert torch.equal(torch.isneginf(ge), ~some), b
        assert ((got - o).abs() <= tol).all(), b
        assert ((ge - e).abs() <= ds + 2.0 ** -22 * (e.abs() + m * 2.0 ** -2))[some].all(), b
