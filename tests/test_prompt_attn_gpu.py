"""Causal attention over packed sequences against its formula in 64 bits."""

import math

import pytest
import torch

from mla_latent_kv_45_b200 import _lib as L
from mla_latent_kv_45_b200 import build
from prompt_testlib import (TINY, V2, attn_inputs, check_attn, dims_of, i32, offsets, run_attn,
                            workspace)

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    L.lib()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def go(dims, new, total, kv, seed=1, spread=1.0):
    cu_q, cu_k = offsets(new), offsets(total)
    t = attn_inputs(dims, cu_q[-1], cu_k[-1], kv, seed, spread)
    out, lse = run_attn(dims, t, cu_q, cu_k)
    check_attn(dims, t, cu_q, cu_k, out, lse)
    return t, out, lse


@pytest.mark.parametrize("n", [1, 2, 16, 17, 63, 64, 65, 115, 127, 128, 129, 200, 255, 256, 257,
                               383, 385, 511, 513, 1000])
def test_one_prompt(n):
    go(dims_of(V2, 2, BF), [n], [n], 2, seed=n)


@pytest.mark.parametrize("n,m", [(1, 1), (1, 64), (1, 127), (1, 128), (1, 129), (1, 5000), (3, 130),
                                 (64, 4097), (128, 1000), (129, 385), (256, 4352), (300, 301),
                                 (257, 2500)])
def test_chunk_behind_cached_rows(n, m):
    go(dims_of(V2, 3, BF), [n], [m], 3, seed=n + m)


@pytest.mark.parametrize("heads,kv", [(1, 1), (4, 1), (4, 2), (6, 2), (6, 3), (5, 5), (12, 1), (24, 2),
                                      (128, 128), (128, 64), (128, 8), (128, 1), (256, 1)])
def test_head_layouts(heads, kv):
    go(dims_of(V2, heads, BF), [70, 1, 190], [70, 150, 200], kv, seed=heads)


@pytest.mark.parametrize("heads,kv", [(8, 1), (16, 1), (64, 1), (128, 1), (6, 1)])
def test_single_tokens_of_grouped_heads(heads, kv):
    """Short chunks of grouped heads behind long prefixes, and heads stored head by head."""
    new, total = [1, 2, 1, 3, 17], [1000, 2, 81, 160, 700]
    dims = dims_of(V2, heads, BF)
    t, out, lse = go(dims, new, total, kv)
    s = {k: (x.transpose(0, 1).contiguous().transpose(0, 1) if x.dim() == 3 else x)
         for k, x in t.items()}
    out2, lse2 = run_attn(dims, s, offsets(new), offsets(total))
    assert torch.equal(out2, out) and torch.equal(lse2, lse)


@pytest.mark.parametrize("new,total,heads,kv", [
    ([1], [9000], 1, 1), ([100], [3000], 2, 2), ([300, 1], [4000, 1], 4, 4),
    ([1, 0, 5, 129], [2000, 700, 3, 129], 8, 8), ([2, 3], [1200, 20000], 16, 1),
    ([700], [100], 1, 1), ([90, 33], [40, 3000], 3, 3), ([1, 1, 1], [1500, 0, 81], 128, 1),
    ([17], [1023], 4, 4), ([17], [1024], 4, 4), ([9000], [9000], 1, 1)])
def test_few_blocks_whose_keys_are_cut(new, total, heads, kv):
    """Fewer blocks than half the multiprocessors: their keys are cut into pieces that are
    merged, beside blocks of one piece, queries that see nothing and empty sequences."""
    go(dims_of(V2, heads, BF), new, total, kv, seed=sum(total))


def test_cut_keys_with_scores_far_apart():
    go(dims_of(V2, 2, BF), [200], [5000], 2, spread=6.0)
    dims = dims_of(V2, 2, BF)
    t = attn_inputs(dims, 40, 4000, 2, 41)
    t["q_nope"] = torch.ones_like(t["q_nope"])
    ramp = torch.linspace(-40, 40, 4000, device="cuda")
    t["k_nope"] = (ramp[:, None, None] / 10 + 0.1 * t["k_nope"].float()).to(BF)
    out, lse = run_attn(dims, t, [0, 40], [0, 4000])
    check_attn(dims, t, [0, 40], [0, 4000], out, lse)


def test_cut_keys_outside_rows_and_bad_offsets():
    dims = dims_of(V2, 2, BF)
    cu_q, cu_k = [3, 20, 90], [100, 2100, 4000]
    t = attn_inputs(dims, 100, 4100, 2, 43)
    for name in ("k_nope", "k_rope", "v"):
        t[name][:100] = math.nan
        t[name][4000:] = math.inf
    ws = workspace(dims, 2, 100)
    out, lse = run_attn(dims, t, cu_q, cu_k, ws=ws)
    check_attn(dims, t, cu_q, cu_k, out, lse)
    for lo, hi in ((0, 3), (90, 100)):
        assert (out[lo:hi] == 7).all() and (lse[lo:hi] == 7).all()
    out2 = torch.full_like(out, 7.0)
    L.mla_prompt_attn(dims, t["q_nope"], t["q_rope"], t["k_nope"], t["k_rope"], t["v"],
                      i32([3, 20, 101]), i32(cu_k), out2, None, ws)
    assert L.mla_get_device_error(ws) == 6
    assert torch.equal(out2[:20], out[:20]) or (out2[20:] == 7).all()
    assert (out2[20:] == 7).all()


def test_cut_keys_give_the_same_bits_every_time():
    dims = dims_of(V2, 4, BF)
    t = attn_inputs(dims, 60, 6000, 4, 45)
    cu_q, cu_k = i32([0, 60]), i32([0, 6000])
    ws = workspace(dims, 1, 60)
    outs = [torch.empty(60, 4, 128, dtype=BF, device="cuda") for _ in range(6)]
    call = lambda o: L.mla_prompt_attn(dims, t["q_nope"], t["q_rope"], t["k_nope"],  # noqa: E731
                                       t["k_rope"], t["v"], cu_q, cu_k, o, None, ws)
    for o in outs[:5]:
        call(o)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(outs[5])
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for o in outs[1:]:
        assert torch.equal(o, outs[0])


def test_packed_lengths_of_every_kind():
    new = [0, 1, 128, 0, 129, 5, 700, 64, 256, 0]
    total = [0, 1, 128, 40, 129, 300, 700, 1000, 257, 0]
    go(dims_of(V2, 4, BF), new, total, 4)


def test_many_sequences():
    new = [(7 * i) % 40 for i in range(400)]
    total = [n + (11 * i) % 90 for i, n in enumerate(new)]
    go(dims_of(V2, 2, BF), new, total, 1)


def test_more_sequences_than_a_block_plans_for_itself():
    new = [(13 * i) % 29 for i in range(700)] + [700]
    total = [n + (5 * i) % 40 for i, n in enumerate(new)]
    go(dims_of(V2, 1, BF), new, total, 1)


@pytest.mark.parametrize("batch,n,heads", [(3, 300, 1), (1200, 300, 1), (60, 2000, 1),
                                           (400, 2000, 2)])
def test_offsets_that_overlap(batch, n, heads):
    """Descending offsets make sequences overlap: more blocks than the tokens have.  The error
    word is set, the workspace is not left, and the next call is right."""
    dims = dims_of(V2, heads, BF)
    t = attn_inputs(dims, n, n, heads, 31)
    size = L.mla_prompt_workspace_size(dims, batch, n)
    whole = torch.full((size + 65536,), 7, dtype=torch.uint8, device="cuda")
    ws = whole[:size]
    L.mla_workspace_init(ws)
    cu = [0, n] * (batch // 2) + [0, n][:batch % 2 + 1]
    out = torch.empty(n, heads, 128, dtype=BF, device="cuda")
    L.mla_prompt_attn(dims, t["q_nope"], t["q_rope"], t["k_nope"], t["k_rope"], t["v"], i32(cu),
                      i32(cu), out, None, ws)
    assert L.mla_get_device_error(ws) == 6
    assert (whole[size:] == 7).all()
    pad = [0] * batch + [n]
    out, lse = run_attn(dims, t, pad, pad, ws=ws)
    check_attn(dims, t, pad, pad, out, lse)


def test_a_workspace_serves_decode_and_prompt_calls_in_turn():
    dims = dims_of(V2, 128, BF)
    size = max(L.mla_workspace_size(dims, 2, 512, 0, 0), L.mla_prompt_workspace_size(dims, 3, 400))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    L.mla_workspace_init(ws)
    g = torch.Generator(device="cuda").manual_seed(3)
    pool = torch.randn(8, 64, 576, generator=g, device="cuda").to(BF)
    cache = L.PagedCache(pool, i32([[0, 3, 5], [1, 2, 6]]), i32([150, 64]))
    q_lat = torch.randn(2, 128, 576, generator=g, device="cuda").to(BF)
    z = [torch.empty(2, 128, 512, dtype=BF, device="cuda") for _ in range(3)]
    new, total = [300, 1, 90], [300, 200, 90]
    t = attn_inputs(dims, sum(new), sum(total), 128, 37)
    for i in range(3):
        L.mla_decode_attn(dims, cache, q_lat, z[i], None, 0, ws)
        assert L.mla_get_device_error(ws) == 0
        out, lse = run_attn(dims, t, offsets(new), offsets(total), ws=ws)
        check_attn(dims, t, offsets(new), offsets(total), out, lse)
    assert torch.equal(z[0], z[1]) and torch.equal(z[0], z[2])


def test_a_workspace_for_many_tokens_does_for_few():
    dims = dims_of(V2, 4, BF)
    ws = workspace(dims, 64, 8192)
    for new, total in (([1], [5000]), ([300, 2], [1500, 2]), ([1] * 64, [90] * 64)):
        t = attn_inputs(dims, sum(new), sum(total), 1, 35)
        out, lse = run_attn(dims, t, offsets(new), offsets(total), ws=ws)
        check_attn(dims, t, offsets(new), offsets(total), out, lse)


def test_refusals_on_the_device():
    dims = dims_of(V2, 2, BF)
    good = attn_inputs(dims, 20, 20, 1, 33)
    ws = workspace(dims, 1, 20)
    out, lse = torch.zeros(20, 2, 128, dtype=BF, device="cuda"), torch.zeros(20, 2, device="cuda")
    cu = i32([0, 20])
    base = dict(good, cu_q=cu, cu_k=cu, out=out, lse=lse, ws=ws)
    L.mla_prompt_attn(dims, **base)
    for name, bad in (("q_nope", good["q_nope"].float()), ("q_nope", good["q_nope"][:, :1]),
                      ("q_rope", good["q_rope"][:19]), ("k_rope", good["k_rope"][:, ::2]),
                      ("k_rope", good["k_rope"].cpu()), ("v", good["v"][:19]),
                      ("v", good["v"].transpose(1, 2)), ("cu_q", cu.long()), ("cu_k", i32([0, 1, 2])),
                      ("out", out.transpose(0, 1)), ("lse", lse.to(BF)), ("lse", lse[:, :1]),
                      ("ws", None), ("ws", ws.cpu())):
        with pytest.raises(ValueError):
            L.mla_prompt_attn(dims, **{**base, name: bad})
    with pytest.raises(L.MlaError) as e:
        L.mla_prompt_attn(dims, **{**base, "ws": ws[:16]})
    assert e.value.status == 4


@pytest.mark.parametrize("batch,heads", [(200, 8), (700, 3), (40, 128)])
def test_many_sequences_without_keys(batch, heads):
    """Queries of many sequences without a key, behind and between sequences that have keys:
    a block without keys may not hold up the block before it."""
    new = [1 + (7 * i) % 30 for i in range(batch)]
    total = [0 if i % 5 else n + i % 90 for i, n in enumerate(new)]
    go(dims_of(V2, heads, BF), new, total, heads)
    go(dims_of(V2, heads, BF), new + [600], [0] * batch + [400], heads)
    # heads in several groups (their keys do not fit L2 together): blocks with keys again
    # behind the blocks without
    go(dims_of(V2, heads, BF), [3] * batch + [60], [0] * batch + [9000], heads)


def test_queries_that_see_no_key():
    """lq > lk: the first lq - lk queries see nothing and get zeros and -inf."""
    new, total = [200, 5, 130, 300], [72, 0, 1, 20]
    go(dims_of(V2, 2, BF), new, total, 2)


def test_no_keys_at_all():
    dims = dims_of(V2, 2, BF)
    t = attn_inputs(dims, 150, 0, 2, 3)
    out, lse = run_attn(dims, t, [0, 100, 150], [0, 0, 0])
    assert (out == 0).all() and torch.isneginf(lse).all()


def test_no_queries():
    dims = dims_of(V2, 2, BF)
    t = attn_inputs(dims, 0, 50, 2, 3)
    out, lse = run_attn(dims, t, [0, 0], [0, 50])
    assert out.numel() == 0


@pytest.mark.parametrize("spread", [3.0, 8.0])
def test_wide_scores(spread):
    """Scores far apart: the running maximum moves by more than a rescale threshold."""
    go(dims_of(V2, 2, BF), [400, 333], [400, 900], 2, spread=spread)


def test_rising_scores_rescale():
    """Every later key outweighs all earlier ones: each tile lifts the maximum."""
    dims = dims_of(V2, 2, BF)
    n = 900
    t = attn_inputs(dims, n, n, 2, 5)
    ramp = torch.linspace(0, 40, n, device="cuda")
    t["q_nope"] = torch.ones_like(t["q_nope"])
    t["k_nope"] = (ramp[:, None, None] / 10 + 0.1 * t["k_nope"].float()).to(BF)
    out, lse = run_attn(dims, t, [0, n], [0, n])
    check_attn(dims, t, [0, n], [0, n], out, lse)


def test_scale_of_the_caller():
    go(dims_of(V2, 2, BF, scale=0.5), [200], [300], 2)


def test_views_of_wider_tensors():
    """Queries and keys as slices of [tokens, heads, 192] and [tokens, heads, 256] products,
    and tensors stored head by head."""
    dims = dims_of(V2, 3, BF)
    new, total = [150, 90], [150, 333]
    cu_q, cu_k = offsets(new), offsets(total)
    t = attn_inputs(dims, cu_q[-1], cu_k[-1], 3, 9)
    ref_out, ref_lse = run_attn(dims, t, cu_q, cu_k)
    q = torch.cat([t["q_nope"], t["q_rope"]], -1)
    kv = torch.cat([t["k_nope"], t["v"]], -1)
    rows = torch.cat([torch.zeros(cu_k[-1], 512, dtype=BF, device="cuda"), t["k_rope"]], -1)
    s = dict(q_nope=q[..., :128], q_rope=q[..., 128:], k_nope=kv[..., :128], v=kv[..., 128:],
             k_rope=rows[:, 512:])
    out, lse = run_attn(dims, s, cu_q, cu_k)
    assert torch.equal(out, ref_out) and torch.equal(lse, ref_lse)
    s = {k: (x.transpose(0, 1).contiguous().transpose(0, 1) if x.dim() == 3 else x)
         for k, x in t.items()}
    out, lse = run_attn(dims, s, cu_q, cu_k)
    assert torch.equal(out, ref_out) and torch.equal(lse, ref_lse)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_what_lies_outside_the_sequences(dtype):
    """NaN and infinities in front of the first sequence, behind the last one and in the next
    sequence's keys reach nothing; rows outside the sequences keep what they held."""
    dims = dims_of(V2, 2, dtype)
    cu_q, cu_k = [5, 75, 205], [9, 109, 259]
    t = attn_inputs(dims, 260, 300, 2, 11)
    for name in ("q_nope", "q_rope"):
        t[name][:5] = math.nan
        t[name][205:] = math.inf
    for name in ("k_nope", "k_rope", "v"):
        t[name][:9] = math.nan
        t[name][259:] = -math.inf
    clean = {k: v.clone() for k, v in t.items()}
    out, lse = run_attn(dims, t, cu_q, cu_k)
    check_attn(dims, t, cu_q, cu_k, out, lse)
    for lo, hi in ((0, 5), (205, 260)):
        assert (out[lo:hi] == 7).all() and (lse[lo:hi] == 7).all()
    for name in ("k_nope", "k_rope", "v"):   # the second sequence's keys turn bad: the first's rows stay
        t[name][109:259] = math.nan
    out2, lse2 = run_attn(dims, t, cu_q, cu_k)
    assert torch.equal(out2[:75], out[:75]) and torch.equal(lse2[:75], lse[:75])
    for name in clean:
        assert clean[name].shape == t[name].shape


def test_later_keys_of_a_sequence_reach_no_earlier_row():
    """Keys that a row does not see may hold anything, values anything finite."""
    dims = dims_of(V2, 2, BF)
    n = 300
    t = attn_inputs(dims, n, n, 2, 13)
    out, lse = run_attn(dims, t, [0, n], [0, n])
    t["k_nope"][200:] = math.nan
    t["v"][200:] = torch.finfo(BF).max
    out2, lse2 = run_attn(dims, t, [0, n], [0, n])
    assert torch.equal(out2[:200], out[:200]) and torch.equal(lse2[:200], lse[:200])


@pytest.mark.parametrize("size,heads,kv", [(TINY, 4, 4), (TINY, 6, 2), (V2, 2, 1),
                                           (dict(d_c=64, d_rope=2, d_nope=5, d_v=3), 3, 3),
                                           (dict(d_c=64, d_rope=128, d_nope=256, d_v=256), 2, 2)])
def test_fp32(size, heads, kv):
    go(dims_of(size, heads, F32), [33, 0, 1, 70, 16], [33, 4, 50, 81, 10], kv)


def test_without_lse():
    dims = dims_of(V2, 2, BF)
    t = attn_inputs(dims, 140, 140, 2, 15)
    want, _ = run_attn(dims, t, [0, 140], [0, 140])
    ws = workspace(dims, 1, 140)
    out = torch.empty_like(want)
    L.mla_prompt_attn(dims, t["q_nope"], t["q_rope"], t["k_nope"], t["k_rope"], t["v"],
                      i32([0, 140]), i32([0, 140]), out, None, ws)
    assert torch.equal(out, want)


def test_bad_offsets_skip_their_sequence():
    """Descending offsets or offsets outside the tensors: the sequence's rows keep what they
    held, the others are computed and the error word is set."""
    dims = dims_of(V2, 2, BF)
    t = attn_inputs(dims, 300, 300, 2, 17)
    ws = workspace(dims, 3, 300)
    for cu_q, cu_k, bad in (([0, 100, 90, 300], [0, 100, 100, 300], slice(90, 90)),
                            ([0, 100, 200, 301], [0, 100, 200, 300], slice(200, 300)),
                            ([0, 100, 200, 300], [0, 100, 200, 400], slice(200, 300)),
                            ([0, 100, 200, 300], [-4, 100, 200, 300], slice(0, 100))):
        out = torch.full((300, 2, 128), 7.0, dtype=BF, device="cuda")
        lse = torch.full((300, 2), 7.0, device="cuda")
        L.mla_prompt_attn(dims, t["q_nope"], t["q_rope"], t["k_nope"], t["k_rope"], t["v"],
                          i32(cu_q), i32(cu_k), out, lse, ws)
        assert L.mla_get_device_error(ws) == 6
        assert (out[bad] == 7).all() and (lse[bad] == 7).all()
        assert L.mla_get_device_error(ws) == 0
    run_attn(dims, t, [0, 100, 200, 300], [0, 100, 200, 300], ws=ws)


def test_same_bits_every_time_and_on_other_streams():
    dims = dims_of(V2, 8, BF)
    new = [300, 17, 513, 128]
    cu = offsets(new)
    t = attn_inputs(dims, cu[-1], cu[-1], 8, 19)
    out, lse = run_attn(dims, t, cu, cu)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    cud = i32(cu)
    bufs = [(workspace(dims, 4, cu[-1]), torch.empty_like(out), torch.empty_like(lse))
            for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, (ws, o, e) in zip((s1, s2), bufs):
            L.mla_prompt_attn(dims, t["q_nope"], t["q_rope"], t["k_nope"], t["k_rope"], t["v"], cud,
                              cud, o, e, ws, s)
            got.append((o, e))
    torch.cuda.synchronize()
    for o, e in got:
        assert torch.equal(o, out) and torch.equal(e, lse)


def test_captured_and_replayed_with_other_lengths():
    """A graph reads the offsets at replay: other lengths within the captured sizes."""
    dims = dims_of(V2, 4, BF)
    t = attn_inputs(dims, 400, 600, 4, 21)
    cu_q, cu_k = i32([0, 400, 400]), i32([0, 600, 600])
    ws = workspace(dims, 2, 400)
    out = torch.empty(400, 4, 128, dtype=BF, device="cuda")
    lse = torch.empty(400, 4, device="cuda")
    call = lambda s=None: L.mla_prompt_attn(dims, t["q_nope"], t["q_rope"], t["k_nope"],  # noqa: E731
                                            t["k_rope"], t["v"], cu_q, cu_k, out, lse, ws, s)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for q, k in (([0, 400, 400], [0, 600, 600]), ([0, 130, 400], [0, 130, 500]),
                 ([0, 1, 300], [0, 40, 600])):
        cu_q.copy_(i32(q))
        cu_k.copy_(i32(k))
        g.replay()
        torch.cuda.synchronize()
        assert L.mla_get_device_error(ws) == 0
        check_attn(dims, t, q, k, out, lse, str(q))


@pytest.mark.parametrize("batch", [127, 128, 129, 300])
def test_fp32_many_sequences(batch):
    """A block finds its sequence 128 at a time."""
    new = [(7 * i + 3 * batch) % 20 for i in range(batch)]
    total = [n + (11 * i) % 30 for i, n in enumerate(new)]
    go(dims_of(TINY, 2, F32), new, total, 1)
    go(dims_of(TINY, 2, F32), [0] * (batch - 1) + [40], [3] * (batch - 1) + [40], 1)


@pytest.mark.parametrize("at", [0, 5, 128, 299])
def test_fp32_bad_offsets_skip_their_sequence(at):
    batch, n = 300, 3
    dims = dims_of(TINY, 2, F32)
    cu = offsets([n] * batch)
    t = attn_inputs(dims, cu[-1], cu[-1], 2, 23)
    ws = workspace(dims, batch, cu[-1])
    want, want_lse = run_attn(dims, t, cu, cu, ws=ws)
    bad_q = list(cu)
    bad_q[at + 1 if at == batch - 1 else at] += 10000 if at == batch - 1 else -10000
    out, lse = torch.full_like(want, 7.0), torch.full_like(want_lse, 7.0)
    L.mla_prompt_attn(dims, t["q_nope"], t["q_rope"], t["k_nope"], t["k_rope"], t["v"],
                      i32(bad_q), i32(cu), out, lse, ws)
    assert L.mla_get_device_error(ws) == 6
    # the sequences on both sides of the bad offset are skipped
    skipped = {at} if at in (0, batch - 1) else {at - 1, at}
    for b in range(batch):
        rows = slice(n * b, n * b + n)
        if b in skipped:
            assert (out[rows] == 7).all() and (lse[rows] == 7).all(), b
        else:
            assert torch.equal(out[rows], want[rows]) and torch.equal(lse[rows], want_lse[rows]), b
    again, _ = run_attn(dims, t, cu, cu, ws=ws)
    assert torch.equal(again, want)
