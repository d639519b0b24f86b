"""Sequences of few queries, which have a kernel of their own, alone and beside long ones."""

import pytest
import torch

from mla_latent_kv_45_b200 import _lib as L
from mla_latent_kv_45_b200 import build
from prompt_testlib import V2, attn_inputs, check_attn, dims_of, i32, offsets, run_attn, workspace

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    L.lib()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def go(new, total, heads, kv, seed=1, spread=1.0):
    dims = dims_of(V2, heads, BF)
    cu_q, cu_k = offsets(new), offsets(total)
    t = attn_inputs(dims, cu_q[-1], cu_k[-1], kv, seed, spread)
    out, lse = run_attn(dims, t, cu_q, cu_k)
    check_attn(dims, t, cu_q, cu_k, out, lse)
    return dims, t, cu_q, cu_k, out, lse


@pytest.mark.parametrize("n", range(1, 18))
def test_tokens(n):
    go([n], [n], 2, 2, seed=n)
    go([n, n, 1], [n + 37, n, 16], 3, 3, seed=n)


@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 255, 257, 1000, 2047])
def test_keys(m):
    go([1, 1], [m, max(1, m - 3)], 2, 1, seed=m)
    # many blocks: the kernel's other shape
    go([1] * 80, [m] + [1 + (7 * i) % min(m, 60) for i in range(79)], 2, 2, seed=m)


@pytest.mark.parametrize("heads,kv", [(2, 1), (3, 1), (5, 1), (16, 1), (17, 1), (12, 4), (6, 2), (16, 16),
                                      (128, 8), (128, 128), (32, 1)])
def test_head_layouts(heads, kv):
    """Rows of a key head from one to more than the kernel takes."""
    rep = heads // kv
    few = max(1, 16 // rep)
    new = [1, few, 0, few + 1, 1, 1, max(1, few - 1), 1]
    go(new, [n + 11 * i for i, n in enumerate(new)], heads, kv, seed=heads)


def test_long_prompts_between_short_ones():
    new = [1] * 60 + [300] + [2] * 60 + [17, 16, 0, 128] + [1] * 60
    total = [n + (29 * i) % 150 for i, n in enumerate(new)]
    go(new, total, 2, 2, seed=5)
    # more sequences than a block plans for itself
    new = [(5 * i) % 4 for i in range(900)] + [500] + [1] * 300
    go(new, [n + (13 * i) % 40 for i, n in enumerate(new)], 1, 1, seed=6)


def test_long_keys_of_many_sequences():
    go([1, 2, 3, 16] * 20, [700 + 13 * i for i in range(80)], 4, 2, seed=8)


def test_queries_that_see_no_key():
    go([16, 5, 1, 3], [4, 0, 0, 3], 2, 2)
    go([16, 5, 1, 3] * 50, [4, 0, 0, 3] * 50, 2, 2)
    dims = dims_of(V2, 2, BF)
    t = attn_inputs(dims, 3, 0, 2, 1)
    out, lse = run_attn(dims, t, [0, 1, 3], [0, 0, 0])
    assert (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("batch", [3, 100])
def test_wide_and_rising_scores(batch):
    go([4] * batch, [90] * batch, 2, 2, spread=6.0)
    dims, t, cu_q, cu_k, _, _ = go([2] * batch, [64] * batch, 2, 1)
    t["k_nope"] *= torch.arange(1, 65, device="cuda").repeat(batch)[:, None, None] / 16
    out, lse = run_attn(dims, t, cu_q, cu_k)
    check_attn(dims, t, cu_q, cu_k, out, lse)


@pytest.mark.parametrize("batch", [4, 100])
def test_what_lies_outside_a_sequence_and_masked_keys(batch):
    """NaN and infinities of other sequences reach nothing; a NaN key reaches only the rows
    that see it, and rows of no sequence are left as they were."""
    dims = dims_of(V2, 2, BF)
    new, total = [3] * batch, [21] * batch
    cu_q, cu_k = offsets(new, 5), offsets(total, 7)
    t = attn_inputs(dims, cu_q[-1] + 6, cu_k[-1] + 4, 2, 3)
    want, want_lse = run_attn(dims, t, cu_q + [cu_q[-1]], cu_k + [cu_k[-1]])
    check_attn(dims, t, cu_q, cu_k, want, want_lse)
    assert (want[:5] == 7).all() and (want[cu_q[-1]:] == 7).all()
    assert (want_lse[:5] == 7).all() and (want_lse[cu_q[-1]:] == 7).all()
    bad = {k: v.clone() for k, v in t.items()}
    for k in ("k_nope", "k_rope", "v"):
        bad[k][:7] = float("nan")
        bad[k][cu_k[2]:cu_k[3]] = float("inf")
        bad[k][cu_k[-1]:] = float("nan")
    out, lse = run_attn(dims, bad, cu_q, cu_k)
    for b in range(batch):
        if b != 2:
            assert torch.equal(out[cu_q[b]:cu_q[b + 1]], want[cu_q[b]:cu_q[b + 1]]), b
            assert torch.equal(lse[cu_q[b]:cu_q[b + 1]], want_lse[cu_q[b]:cu_q[b + 1]]), b
    # the last key of sequence 1: only its last query sees it
    one = {k: v.clone() for k, v in t.items()}
    one["k_nope"][cu_k[2] - 1] = float("nan")
    one["v"][cu_k[2] - 1] = torch.finfo(BF).max
    out, lse = run_attn(dims, one, cu_q, cu_k)
    last = cu_q[2] - 1
    assert torch.isnan(out[last]).all() and torch.isnan(lse[last]).all()
    out[last], lse[last] = want[last], want_lse[last]
    assert torch.equal(out[5:cu_q[-1]], want[5:cu_q[-1]])


def test_views_of_wider_tensors():
    dims = dims_of(V2, 4, BF)
    g = torch.Generator(device="cuda").manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)  # noqa: E731
    q, kv, rows = r(9, 4, 200), r(80, 2, 264), r(80, 576)
    t = dict(q_nope=q[..., :128], q_rope=q[..., 136:], k_nope=kv[..., :128], v=kv[..., 136:],
             k_rope=rows[:, 512:])
    out, lse = run_attn(dims, t, [0, 2, 8, 9], [0, 20, 50, 80])
    check_attn(dims, t, [0, 2, 8, 9], [0, 20, 50, 80], out, lse)


def test_bad_offsets_skip_their_sequence():
    dims = dims_of(V2, 2, BF)
    n = 40
    cu = offsets([3] * n)
    t = attn_inputs(dims, cu[-1], cu[-1], 2, 9)
    ws = workspace(dims, n, cu[-1])
    want, _ = run_attn(dims, t, cu, cu, ws=ws)
    for which in (0, 1):
        bad = list(cu)
        bad[20] += 100000
        out = torch.full_like(want, 7.0)
        both = [cu, cu]
        both[which] = bad
        L.mla_prompt_attn(dims, t["q_nope"], t["q_rope"], t["k_nope"], t["k_rope"], t["v"],
                          i32(both[0]), i32(both[1]), out, None, ws)
        assert L.mla_get_device_error(ws) == 6
        assert (out[57:63] == 7).all()
        assert torch.equal(out[:57], want[:57]) and torch.equal(out[63:], want[63:])


def test_captured_and_replayed_with_other_lengths():
    """One captured call whose sequences are short in one replay and long in the next."""
    dims = dims_of(V2, 2, BF)
    n_q, n_k, batch = 320, 900, 40
    t = attn_inputs(dims, n_q, n_k, 2, 12)
    ws = workspace(dims, batch, n_q)
    cu_q, cu_k = i32([0] * (batch + 1)), i32([0] * (batch + 1))
    out = torch.zeros(n_q, 2, 128, dtype=BF, device="cuda")
    lse = torch.zeros(n_q, 2, device="cuda")
    call = lambda: L.mla_prompt_attn(dims, t["q_nope"], t["q_rope"], t["k_nope"], t["k_rope"],  # noqa: E731
                                     t["v"], cu_q, cu_k, out, lse, ws)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for new in ([8] * 40, [320] + [0] * 39, [1] * 39 + [200], [16, 17] * 9 + [0] * 22):
        total = [n + 5 for n in new]
        q, k = offsets(new), offsets(total)
        cu_q.copy_(i32(q))
        cu_k.copy_(i32(k))
        first = None
        for _ in range(3):
            out.fill_(7)
            g.replay()
            assert L.mla_get_device_error(ws) == 0
            first = out.clone() if first is None else first
            assert torch.equal(out, first)
        check_attn(dims, t, q, k, out, lse)
        assert (out[q[-1]:] == 7).all()


@pytest.mark.parametrize("long", [0, 17, 200])
def test_beside_blocks_whose_keys_are_cut(long):
    """Few blocks over more than 1024 keys: those that the other kernel leaves are cut and
    joined, and where it leaves none the join finds nothing to do."""
    new, total = [1, 2, 16] * 7 + [long], [60] * 21 + [long + 300 if long else 0]
    dims, t, cu_q, cu_k, out, lse = go(new, total, 2, 2, seed=long)
    ws = workspace(dims, 22, cu_q[-1])
    for _ in range(3):
        again, lse2 = run_attn(dims, t, cu_q, cu_k, ws=ws)
        assert torch.equal(again, out) and torch.equal(lse2, lse)
    # the same workspace for a call that is cut, then for one that is not
    go([64], [1500], 2, 2)
    big = attn_inputs(dims, 64, 1500, 2, 5)
    o, e = run_attn(dims, big, [0, 64], [0, 1500], ws=ws)
    check_attn(dims, big, [0, 64], [0, 1500], o, e)
    again, lse2 = run_attn(dims, t, cu_q, cu_k, ws=ws)
    assert torch.equal(again, out) and torch.equal(lse2, lse)
