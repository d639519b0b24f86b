"""Plain 64-bit implementations of the prompt operators and their inputs, for the tests.

Tolerances count roundings; a rounding to type t is off by at most half a step,
finfo(t).eps / 2 relative to the value.
"""

from __future__ import annotations

import math

import torch

from mla_latent_kv_45_b200 import _lib as L

V2 = dict(d_c=512, d_rope=64, d_nope=128, d_v=128)
TINY = dict(d_c=16, d_rope=8, d_nope=8, d_v=8)


def dims_of(size, heads, dtype, page=64, layout=L.MLA_ROPE_INTERLEAVED, cache=L.MLA_CACHE_NATIVE,
            scale=0.0):
    return L.Dims(heads, size["d_c"], size["d_rope"], size["d_nope"], size["d_v"], page,
                  L.MLA_BF16 if dtype == torch.bfloat16 else L.MLA_FP32, layout, 10000.0, 1e-6,
                  scale, cache)


def offsets(lens, first=0):
    out = [first]
    for n in lens:
        out.append(out[-1] + n)
    return out


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def workspace(dims, batch, tokens):
    ws = torch.empty(L.mla_prompt_workspace_size(dims, batch, tokens), dtype=torch.uint8,
                     device="cuda")
    L.mla_workspace_init(ws)
    return ws


# ---------------------------------------------------------------- attention


def attn_inputs(dims, n_q, n_k, kv, seed, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: (spread * torch.randn(*s, generator=g, device="cuda")).to(dims.torch_dtype)  # noqa: E731
    return dict(q_nope=r(n_q, dims.n_heads, dims.d_nope), q_rope=r(n_q, dims.n_heads, dims.d_rope),
                k_nope=r(n_k, kv, dims.d_nope), k_rope=r(n_k, dims.d_rope), v=r(n_k, kv, dims.d_v))


def attn_ref(dims, t, cu_q, cu_k):
    """Yields (rows of the packed queries, out, lse, weights . |v|, largest sum of |q k|) per
    sequence, in 64 bits; the last two carry the tolerance."""
    scale = dims.softmax_scale or 1.0 / math.sqrt(dims.d_nope + dims.d_rope)
    rep = dims.n_heads // t["k_nope"].shape[1]
    for b in range(len(cu_q) - 1):
        q0, q1, k0, k1 = cu_q[b], cu_q[b + 1], cu_k[b], cu_k[b + 1]
        n, m = q1 - q0, k1 - k0
        q = torch.cat([t["q_nope"][q0:q1], t["q_rope"][q0:q1]], -1).double().transpose(0, 1)
        kr = t["k_rope"][k0:k1, None].expand(-1, t["k_nope"].shape[1], -1)
        k = torch.cat([t["k_nope"][k0:k1], kr], -1).double().transpose(0, 1)
        k = k.repeat_interleave(rep, 0)
        v = t["v"][k0:k1].double().transpose(0, 1).repeat_interleave(rep, 0)
        seen = (torch.arange(m, device="cuda")[None]
                <= torch.arange(n, device="cuda")[:, None] + m - n)
        x = (q @ k.transpose(1, 2)) * scale
        size = (q.abs() @ k.abs().transpose(1, 2)) * scale
        x = x.masked_fill(~seen, -math.inf)
        lse = torch.logsumexp(x, -1) if m else torch.full(x.shape[:2], -math.inf,
                                                          dtype=torch.float64, device="cuda")
        p = torch.exp(x - lse[..., None]).masked_fill(~seen, 0.0)
        o, a = p @ v, p @ v.abs()
        big = size.masked_fill(~seen, 0.0).amax(-1) if m else torch.zeros_like(lse)
        yield (slice(q0, q1), o.transpose(0, 1), lse.transpose(0, 1), a.transpose(0, 1),
               big.transpose(0, 1))


def check_attn(dims, t, cu_q, cu_k, out, lse, what=""):
    """bf16: the weights are rounded once (2^-8 of A = sum p |v| / l) and the result once (2^-8
    of |out|).  A score is a sum of d products in 32 bits, each addition off by at most 2^-23 of
    the running sum (a tensor core may truncate), so it is within d 2^-23 of max sum |q k|;
    that moves a weight, the sum and lse by the same amount.  The exponential is within 2^-17.
    fp32: no rounded weights; the sum over n keys adds n 2^-24."""
    d = dims.d_nope + dims.d_rope
    bf = dims.torch_dtype == torch.bfloat16
    for b, (rows, o, e, a, big) in enumerate(attn_ref(dims, t, cu_q, cu_k)):
        if o.numel() == 0:
            continue
        n = cu_k[b + 1] - cu_k[b]
        ds = d * 2.0 ** -23 * big + (2.0 ** -17 if bf else 2.0 ** -21)
        some = torch.isfinite(e)
        got, ge = out[rows].double(), lse[rows].double()
        assert torch.equal(torch.isneginf(ge), ~some), (what, b)
        assert (got[~some] == 0).all(), (what, b)
        tol = 2 * ds[..., None] * a + 2.0 ** -24 * (n + 8) * a
        if bf:
            tol = tol + 2.0 ** -8 * (a + o.abs())
        bad = ((got - o).abs() > tol) & some[..., None]
        bad |= ~torch.isfinite(got)
        assert not bad.any(), (what, b, int(bad.sum()), float(((got - o).abs() - tol)[bad].max()))
        tl = ds + 2.0 ** -22 * (e.abs() + n * 2.0 ** -2)
        off = ((ge - e).abs() > tl) & some
        assert not off.any(), (what, b, "lse", float((ge - e).abs()[some].max()))


def run_attn(dims, t, cu_q, cu_k, ws=None, out=None, lse=None, stream=None):
    n_q = t["q_nope"].shape[0]
    ws = workspace(dims, len(cu_q) - 1, n_q) if ws is None else ws
    out = torch.full((n_q, dims.n_heads, dims.d_v), 7.0, dtype=dims.torch_dtype,
                     device="cuda") if out is None else out
    lse = torch.full((n_q, dims.n_heads), 7.0, device="cuda") if lse is None else lse
    L.mla_prompt_attn(dims, t["q_nope"], t["q_rope"], t["k_nope"], t["k_rope"], t["v"], i32(cu_q),
                      i32(cu_k), out, lse, ws, stream)
    assert L.mla_get_device_error(ws, stream) == 0
    return out, lse


# ---------------------------------------------------------------- cache rows


def rotate_ref(x, pos, layout):
    d = x.shape[-1]
    x = x.double()
    i = torch.arange(d // 2, device=x.device)
    ang = pos.double()[:, None] * 10000.0 ** (-2.0 * i.double() / d)
    if x.dim() == 3:
        ang = ang[:, None]
    j0, j1 = (i, i + d // 2) if layout == L.MLA_ROPE_HALF else (2 * i, 2 * i + 1)
    a, b = x[..., j0], x[..., j1]
    out, size = torch.empty_like(x), torch.empty_like(x)
    out[..., j0] = a * torch.cos(ang) - b * torch.sin(ang)
    out[..., j1] = a * torch.sin(ang) + b * torch.cos(ang)
    size[..., j0] = size[..., j1] = a.abs() + b.abs()
    return out, size


def close_rotated(got, ref, size, dtype):
    """cos and sin are within 2^-21, two products and a sum in 32 bits; then one rounding."""
    tol = 2.0 ** -20 * size + (torch.finfo(dtype).eps / 2) * ref.abs() * (1 + 2.0 ** -10)
    return bool(((got.double() - ref).abs() <= tol).all())


def norm_ref(x, gamma):
    x = x.double()
    return gamma.double() * x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)


def close_normed(got, ref, d_c, dtype):
    """A sum of d_c squares in 32 bits (d_c 2^-24 at most, halved by the root), four more
    operations, then one rounding."""
    rel = (d_c / 2 + 8) * 2.0 ** -24 + (torch.finfo(dtype).eps / 2 if dtype != torch.float32 else 0)
    return bool(((got.double() - ref).abs() <= rel * ref.abs() * (1 + 2.0 ** -10)).all())


def paged(dims, lens, seed, spare=3, extra_pages=0):
    """A shuffled pool full of rows and a page table; unused table entries are -1."""
    g = torch.Generator().manual_seed(seed)
    page = dims.page_size
    need = [-(-n // page) for n in lens]
    num = sum(need) + spare
    order = torch.randperm(num, generator=g)
    table = torch.full((len(lens), max(need + [1]) + extra_pages), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    if dims.cache_format == L.MLA_CACHE_INT8:
        pool = torch.zeros(num, page, 656, dtype=torch.uint8)
        pool[..., :512] = torch.randint(-127, 128, (num, page, 512), generator=g,
                                        dtype=torch.int16).to(torch.int8).view(torch.uint8)
        pool[..., 512:640] = torch.randn(num, page, 64, generator=g).to(torch.bfloat16).view(torch.uint8)
        e = torch.randint(-9, 3, (num, page, 1), generator=g)
        pool[..., 640:644] = torch.exp2(e.float()).view(torch.uint8)
    else:
        pool = torch.randn(num, page, dims.d_c + dims.d_rope, generator=g).to(dims.torch_dtype)
    return L.PagedCache(pool.cuda(), table.cuda(), None)


def row_values(dims, raw):
    """The values [c ; k_R] of raw pool rows (exact)."""
    if dims.cache_format != L.MLA_CACHE_INT8:
        return raw.double()
    c = raw[..., :512].contiguous().view(torch.int8).double()
    s = raw[..., 640:644].contiguous().view(torch.float32).double()
    return torch.cat([c * s, raw[..., 512:640].contiguous().view(torch.bfloat16).double()], -1)


def rows_of(cache, b, first, n, page):
    pos = torch.arange(first, first + n, device="cuda")
    return cache.pool[cache.block_table[b].long()[pos // page], pos % page]
