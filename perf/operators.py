"""Measured cases of the prompt operators of a Multi-head Latent Attention layer.

Three operators carry a prompt (or a chunk of one) through the layer: the
append that normalises, rotates and writes the rows of many new tokens into the
paged latent cache and rotates their queries, the gather that reads a
sequence's rows back out of the pages, and causal attention over packed
sequences with keys and values that were expanded per head.

With ``own`` false ``run`` computes them in elementary torch operations; with
``own`` true it makes the library's calls.  ``exact`` computes the same outputs
in 64 bits, sequence by sequence, from the definitions.

Fields of a case: ``op``; ``batch`` sequences whose new-token counts are drawn
from ``new_min .. new_max`` and whose already cached rows from ``ctx_min ..
ctx_max`` (by ``lens_seed``); ``heads`` query heads and ``kv_heads`` key heads;
``size`` ("v2": 512 latent + 64 rotated values per row, 128-wide heads;
"tiny": 16 + 8, 8-wide heads); ``dtype``; ``cache`` ("native" or "int8" rows);
``layout`` of the rotated pairs.
"""

import math
import random

import torch

own = False

SIZES = {
    # d_c, d_rope, d_nope, d_v, page_size
    "v2": (512, 64, 128, 128, 64),
    "tiny": (16, 8, 8, 8, 16),
}
ROPE_BASE, RMS_EPS = 10000.0, 1e-6


def _case(name, op, batch, new_min, new_max, ctx_min, ctx_max, heads=128, kv_heads=0, size="v2",
          dtype="bf16", cache="native", layout="interleaved", lens_seed=7):
    c = dict(op=op, batch=batch, new_min=new_min, new_max=new_max, ctx_min=ctx_min,
             ctx_max=ctx_max, heads=heads, kv_heads=kv_heads or heads, size=size, dtype=dtype,
             cache=cache, layout=layout, lens_seed=lens_seed)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one short question: latency, a single ragged tile per head
        _case("attn_115", "attn", 1, 115, 115, 0, 0),
        # one long document in a single pass: the tensor-core rate
        _case("attn_8192", "attn", 1, 8192, 8192, 0, 0),
        # a serving batch of prompts packed back to back, lengths from a word to a page
        _case("attn_packed", "attn", 16, 1, 2048, 0, 0),
        # a chunk of 256 tokens over 4096 cached rows (chunked prefill)
        _case("attn_chunk256", "attn", 1, 256, 256, 4096, 4096),
        # grouped heads, several sequences with prefixes of their own
        _case("attn_grouped", "attn", 4, 512, 2048, 0, 2048, kv_heads=8),
        # the 32-bit validation sizes
        _case("attn_fp32_tiny", "attn", 2, 33, 33, 0, 0, heads=4, size="tiny", dtype="fp32"),
        # a long document's rows and queries
        _case("append_8192", "append", 1, 8192, 8192, 0, 0),
        # the chunks of a serving batch, each behind the rows its sequence already has
        _case("append_ragged", "append", 32, 1, 512, 0, 8192, layout="half"),
        # a chunk appended to 8-bit rows and the whole sequence read back, as chunked prefill does
        _case("append_int8", "append", 1, 256, 256, 4096, 4096, cache="int8"),
        # one sequence's prefix
        _case("gather_4352", "gather", 1, 256, 256, 4096, 4096),
        # the prefixes of a whole batch
        _case("gather_batch64", "gather", 64, 1, 1, 1024, 8192),
        # a very long prefix in 8-bit rows
        _case("gather_long_int8", "gather", 1, 1, 1, 131071, 131071, cache="int8"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


MOST_PAIRS = 128 * 8192 * 8193 // 2     # head-query-key triples of the largest listed attention
MOST_ROWS = 256 * 1024                  # rows of the largest listed gather
MOST_TOKENS = 8192                      # new tokens of the largest listed append


def draw(rng):
    op = rng.choice(["attn", "attn", "append", "gather"])
    layout = rng.choice(["interleaved", "half"])
    seed = rng.randrange(1 << 30)
    while True:
        batch = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, 8192)
        lo = rng.randint(1, hi)
        chi = rng.choice([0, _log_int(rng, 1, 8192)])
        clo = rng.randint(0, chi)
        if op == "attn":
            heads = rng.choice([1, 2, 4, 8, 16, 32, 64, 128, 128])
            kv = rng.choice([h for h in (1, 2, 4, 8, 16, 32, 64, 128) if heads % h == 0] + [heads])
            if rng.random() < 0.15:     # the 32-bit path is for validation: small sizes
                heads = min(heads, 8)
                kv = math.gcd(kv, heads)
                c = _case("", op, min(batch, 4), min(lo, 64), min(hi, 64), min(clo, 64),
                          min(chi, 64), heads, kv, "tiny", "fp32", "native", layout, seed)
            else:
                c = _case("", op, batch, lo, hi, clo, chi, heads, kv, "v2", "bf16", "native",
                          layout, seed)
            new, ctx = _lens(c)
            if heads * sum(n * x + n * (n + 1) // 2 for n, x in zip(new, ctx)) > MOST_PAIRS:
                continue
            if sum(new) + sum(ctx) > 65536:
                continue
            return c
        if op == "append":
            if rng.random() < 0.15:
                return _case("", op, min(batch, 4), min(lo, 64), min(hi, 64), min(clo, 64),
                             min(chi, 64), 4, 4, "tiny", "fp32", "native", layout, seed)
            c = _case("", op, batch, lo, hi, clo, chi, rng.choice([16, 32, 64, 128, 128]), 0, "v2",
                      "bf16", rng.choice(["native", "int8"]), layout, seed)
            new, ctx = _lens(c)
            if sum(new) > MOST_TOKENS or sum(ctx) > MOST_ROWS // 2:
                continue
            return c
        c = _case("", op, batch, lo, hi, clo, chi, 128, 0, "v2", "bf16",
                  rng.choice(["native", "int8"]), layout, seed)
        new, ctx = _lens(c)
        if sum(new) + sum(ctx) > MOST_ROWS:
            continue
        return c


def _lens(case):
    """New tokens and already cached rows of each sequence."""
    r = random.Random(case["lens_seed"])
    new = [r.randint(case["new_min"], case["new_max"]) for _ in range(case["batch"])]
    ctx = [r.randint(case["ctx_min"], case["ctx_max"]) for _ in range(case["batch"])]
    return new, ctx


def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _offsets(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _inputs(case, seed):
    """The inputs of a case, made on the GPU from the seed alone."""
    d_c, d_r, d_n, d_v, page = SIZES[case["size"]]
    new, ctx = _lens(case)
    total = [a + b for a, b in zip(new, ctx)]
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = _type(case)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda").to(t)  # noqa: E731
    s = dict(new=new, ctx=ctx, total=total)
    s["cu_new"], s["cu_all"], s["ctx_lens"] = i32(_offsets(new)), i32(_offsets(total)), i32(ctx)
    H, KV, Tq, Tk = case["heads"], case["kv_heads"], sum(new), sum(total)
    if case["op"] == "attn":
        s["q_nope"], s["q_rope"] = randn(Tq, H, d_n), randn(Tq, H, d_r)
        s["k_nope"], s["k_rope"], s["v"] = randn(Tk, KV, d_n), randn(Tk, d_r), randn(Tk, KV, d_v)
        return s
    # a paged pool in shuffled page order that already holds rows everywhere
    need = [-(-n // page) for n in total]
    pages = sum(need) + 8
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(case["batch"], max(need), dtype=torch.int32)
    order, at = order.cpu(), 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    s["table"] = table.cuda()
    if case["cache"] == "int8":
        codes = torch.randint(-127, 128, (pages, page, d_c), generator=g, device="cuda",
                              dtype=torch.int16).to(torch.int8)
        pool = torch.zeros(pages, page, 656, dtype=torch.uint8, device="cuda")
        pool[..., :512] = codes.view(torch.uint8)
        pool[..., 512:640] = randn(pages, page, d_r).view(torch.uint8)
        e = torch.randint(-6, -3, (pages, page, 1), generator=g, device="cuda")
        pool[..., 640:644] = torch.exp2(e.float()).view(torch.uint8)
        s["pool"] = pool
    else:
        s["pool"] = randn(pages, page, d_c + d_r)
    if case["op"] == "append":
        # raw projections of unit-variance hidden states with N(0, 0.02^2) weights
        s["x"] = (1.4 * torch.randn(Tq, d_c + d_r, generator=g, device="cuda")).to(t)
        s["gamma"] = (1 + 0.1 * torch.randn(d_c, generator=g, device="cuda")).to(t)
        s["q_rope"] = randn(Tq, H, d_r)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    d_c, d_r, d_n, d_v, page = SIZES[case["size"]]
    if own:
        # the handles and output buffers a serving loop keeps
        from mla_latent_kv_45_b200 import _lib as L
        s["dims"] = L.Dims(case["heads"], d_c, d_r, d_n, d_v, page,
                           L.MLA_BF16 if case["dtype"] == "bf16" else L.MLA_FP32,
                           L.MLA_ROPE_HALF if case["layout"] == "half" else L.MLA_ROPE_INTERLEAVED,
                           ROPE_BASE, RMS_EPS, 0.0,
                           L.MLA_CACHE_INT8 if case["cache"] == "int8" else L.MLA_CACHE_NATIVE)
        Tq, Tk, t = sum(s["new"]), sum(s["total"]), _type(case)
        nbytes = L.mla_prompt_workspace_size(s["dims"], case["batch"], Tq)
        s["ws"] = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        L.mla_workspace_init(s["ws"])
        if case["op"] == "attn":
            s["out"] = torch.empty(Tq, case["heads"], d_v, dtype=t, device="cuda")
            s["lse"] = torch.empty(Tq, case["heads"], dtype=torch.float32, device="cuda")
        else:
            s["cache"] = L.PagedCache(s["pool"], s["table"], None)
            s["rows"] = torch.empty(Tk, d_c + d_r, dtype=t, device="cuda")
            if case["op"] == "append":
                s["q_out"] = torch.empty_like(s["q_rope"])
    return s


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from mla_latent_kv_45_b200 import _lib as L
    case = s["case"]
    if case["op"] == "attn":
        L.mla_prompt_attn(s["dims"], s["q_nope"], s["q_rope"], s["k_nope"], s["k_rope"], s["v"],
                          s["cu_new"], s["cu_all"], s["out"], s["lse"], s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    if case["op"] == "gather":
        L.mla_cache_gather(s["dims"], s["cache"], s["cu_all"], None, s["rows"], s["ws"])
        return {"rows": s["rows"]}
    L.mla_prompt_append(s["dims"], s["cache"], s["x"], s["gamma"], s["cu_new"], s["ctx_lens"],
                        s["q_rope"], s["q_out"], s["ws"])
    if case["cache"] == "int8":
        L.mla_cache_gather(s["dims"], s["cache"], s["cu_all"], None, s["rows"], s["ws"])
        return {"rows": s["rows"], "q": s["q_out"]}
    return {"pool": s["pool"], "q": s["q_out"]}


# ------------------------------------------------------------------ plain form


def _plain_attn(s):
    case = s["case"]
    d_c, d_r, d_n, d_v, _ = SIZES[case["size"]]
    H, KV, t = case["heads"], case["kv_heads"], _type(case)
    scale = 1.0 / math.sqrt(d_n + d_r)
    out = torch.empty(sum(s["new"]), H, d_v, dtype=t, device="cuda")
    lse = torch.empty(sum(s["new"]), H, dtype=torch.float32, device="cuda")
    q0 = k0 = 0
    for n, m in zip(s["new"], s["total"]):
        seen = (torch.arange(m, device="cuda")[None, :]
                <= torch.arange(n, device="cuda")[:, None] + (m - n))
        kr = s["k_rope"][k0:k0 + m].float()
        step = max(1, (1 << 28) // (n * m))
        for h0 in range(0, H, step):
            hs = torch.arange(h0, min(H, h0 + step), device="cuda")
            ks = hs // (H // KV)
            q = s["q_nope"][q0:q0 + n].index_select(1, hs).float().transpose(0, 1)
            qr = s["q_rope"][q0:q0 + n].index_select(1, hs).float().transpose(0, 1)
            k = s["k_nope"][k0:k0 + m].index_select(1, ks).float().permute(1, 2, 0)
            v = s["v"][k0:k0 + m].index_select(1, ks).float().transpose(0, 1)
            x = (q @ k + qr @ kr.T) * scale
            x = torch.where(seen, x, -math.inf)
            top = x.amax(-1, keepdim=True)
            p = torch.exp(x - top)
            l = p.sum(-1, keepdim=True)
            out[q0:q0 + n, h0:h0 + len(hs)] = ((p @ v) / l).transpose(0, 1).to(t)
            lse[q0:q0 + n, h0:h0 + len(hs)] = (top + torch.log(l))[..., 0].T
        q0, k0 = q0 + n, k0 + m
    return {"out": out, "lse": lse}


def _slots(table, lens, starts, page):
    """Flat pool row of every token of the packed sequences."""
    seq = torch.repeat_interleave(torch.arange(len(lens), device="cuda"),
                                  torch.tensor(lens, device="cuda"))
    first = torch.tensor(_offsets(lens)[:-1], device="cuda")
    pos = torch.arange(sum(lens), device="cuda") - first[seq] + torch.tensor(starts, device="cuda")[seq]
    return table.long()[seq, pos // page] * page + pos % page, pos


def _rotate(x, pos, case):
    """Pairs of x's last axis rotated by the token's position (angles in 64 bits)."""
    d = x.shape[-1]
    theta = ROPE_BASE ** (-torch.arange(0, d, 2, dtype=torch.float64, device="cuda") / d)
    a = pos.double()[:, None] * theta
    cos, sin = torch.cos(a).float(), torch.sin(a).float()
    if x.dim() == 3:
        cos, sin = cos[:, None], sin[:, None]
    if case["layout"] == "half":
        x0, x1 = x[..., :d // 2], x[..., d // 2:]
        return torch.cat([x0 * cos - x1 * sin, x0 * sin + x1 * cos], -1)
    x0, x1 = x[..., 0::2], x[..., 1::2]
    return torch.stack([x0 * cos - x1 * sin, x0 * sin + x1 * cos], -1).flatten(-2)


def _pow2_scale(c):
    """Smallest power of two s with max |c| <= 127 s for each row (0 rows: 1)."""
    top = c.abs().amax(-1, keepdim=True)
    e = torch.frexp(top)[1] - 7
    e = torch.where(top > 127 * torch.exp2(e.double()), e + 1, e)
    return torch.exp2(torch.where(top > 0, e, torch.zeros_like(e)).double())


def _plain_rows(s):
    case = s["case"]
    t = _type(case)
    d_c, d_r, _, _, page = SIZES[case["size"]]
    slot, _ = _slots(s["table"], s["total"], [0] * case["batch"], page)
    if case["cache"] == "native":
        return s["pool"].view(-1, d_c + d_r)[slot]
    raw = s["pool"].view(-1, 656)[slot]
    scale = raw[:, 640:644].contiguous().view(torch.float32)
    c = raw[:, :512].contiguous().view(torch.int8).float() * scale
    return torch.cat([c.to(t), raw[:, 512:640].contiguous().view(t)], -1)


def _plain_append(s):
    case = s["case"]
    t = _type(case)
    d_c, d_r, _, _, page = SIZES[case["size"]]
    slot, pos = _slots(s["table"], s["new"], s["ctx"], page)
    # 64 bits for 8-bit rows: codes next to a border between two steps
    wide = torch.float64 if case["cache"] == "int8" else torch.float32
    x, gamma = s["x"][:, :d_c].to(wide), s["gamma"].to(wide)
    c = gamma * x / torch.sqrt((x * x).mean(-1, keepdim=True) + RMS_EPS)
    k = _rotate(s["x"][:, d_c:].float(), pos, case).to(t)
    q = _rotate(s["q_rope"].float(), pos, case).to(t)
    if case["cache"] == "native":
        s["pool"].view(-1, d_c + d_r)[slot] = torch.cat([c.to(t), k], -1)
        return {"pool": s["pool"], "q": q}
    scale = _pow2_scale(c)
    codes = torch.round(c / scale).clamp(-127, 127).to(torch.int8)
    row = torch.zeros(len(slot), 656, dtype=torch.uint8, device="cuda")
    row[:, :512] = codes.view(torch.uint8)
    row[:, 512:640] = k.contiguous().view(torch.uint8)
    row[:, 640:644] = scale.float().view(torch.uint8)
    s["pool"].view(-1, 656)[slot] = row
    return {"rows": _plain_rows(s), "q": q}


def _run_plain(s):
    op = s["case"]["op"]
    if op == "attn":
        return _plain_attn(s)
    if op == "gather":
        return {"rows": _plain_rows(s)}
    return _plain_append(s)


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    d_c, d_r, d_n, d_v, page = SIZES[case["size"]]
    new, ctx = _lens(case)
    H, KV = case["heads"], case["kv_heads"]
    b = 2 if case["dtype"] == "bf16" else 4
    Tq, Tk = sum(new), sum(new) + sum(ctx)
    row = 644 if case["cache"] == "int8" else (d_c + d_r) * b
    wide = (d_c + d_r) * b
    if case["op"] == "attn":
        pairs = sum(n * x + n * (n + 1) // 2 for n, x in zip(new, ctx))
        return {"bytes": b * (Tq * H * (d_n + d_r + d_v) + Tk * (KV * (d_n + d_v) + d_r)) + 4 * Tq * H,
                "flops": 2.0 * H * pairs * (d_n + d_r + d_v)}
    if case["op"] == "gather":
        return {"bytes": Tk * (row + wide), "flops": 0}
    append = Tq * (wide + row + 2 * H * d_r * b)
    if case["cache"] == "int8":
        append += Tk * (row + wide)
    return {"bytes": append, "flops": 3.0 * Tq * (2 * d_c + (H + 1) * d_r)}


# ------------------------------------------------------------------ 64 bits, from the definitions


def exact(case, seed):
    s = _inputs(case, seed)
    d_c, d_r, d_n, d_v, page = SIZES[case["size"]]
    H, KV = case["heads"], case["kv_heads"]
    if case["op"] == "attn":
        outs, lses, q0, k0 = [], [], 0, 0
        for n, m in zip(s["new"], s["total"]):
            o = torch.empty(n, H, d_v, dtype=torch.float64, device="cuda")
            e = torch.empty(n, H, dtype=torch.float64, device="cuda")
            first = m - n
            for h in range(H):
                j = h * KV // H
                q = torch.cat([s["q_nope"][q0:q0 + n, h], s["q_rope"][q0:q0 + n, h]], -1).double()
                k = torch.cat([s["k_nope"][k0:k0 + m, j], s["k_rope"][k0:k0 + m]], -1).double()
                x = torch.einsum("id,jd->ij", q, k).div_(math.sqrt(d_n + d_r))
                x += torch.full((n, m), -math.inf, dtype=torch.float64, device="cuda").triu_(first + 1).nan_to_num_(nan=0.0, neginf=-math.inf)
                e[:, h] = torch.logsumexp(x, -1)
                o[:, h] = x.sub_(e[:, h, None]).exp_() @ s["v"][k0:k0 + m, j].double()
            outs.append(o)
            lses.append(e)
            q0, k0 = q0 + n, k0 + m
        return {"out": torch.cat(outs), "lse": torch.cat(lses)}

    def turned(x, positions):
        """e^(i pos theta) times the pairs as complex numbers."""
        d = x.shape[-1]
        x = x.double()
        z = (torch.complex(x[..., :d // 2], x[..., d // 2:]) if case["layout"] == "half"
             else torch.complex(x[..., 0::2], x[..., 1::2]))
        th = torch.tensor([ROPE_BASE ** (-2.0 * i / d) for i in range(d // 2)],
                          dtype=torch.float64, device="cuda")
        a = torch.outer(positions.double(), th)
        w = torch.polar(torch.ones_like(a), a)
        z = z * (w if z.dim() == 2 else w.unsqueeze(1))
        return (torch.cat([z.real, z.imag], -1) if case["layout"] == "half"
                else torch.view_as_real(z).reshape(x.shape))

    if case["cache"] == "int8":
        held = s["pool"][..., :512].contiguous().view(torch.int8).double()
        held = held * s["pool"][..., 640:644].contiguous().view(torch.float32).double()
        pool = torch.cat([held, s["pool"][..., 512:640].contiguous().view(torch.bfloat16).double()], -1)
    else:
        pool = s["pool"].double()
    q_all, t0 = [], 0
    for b in range(case["batch"]):
        if case["op"] == "gather":
            break
        n, p0 = s["new"][b], s["ctx"][b]
        pos = torch.arange(p0, p0 + n, device="cuda")
        x = s["x"][t0:t0 + n].double()
        c = x[:, :d_c]
        c = s["gamma"].double() * c * (c.pow(2).sum(-1, keepdim=True) / d_c + RMS_EPS).rsqrt()
        if case["cache"] == "int8":
            top = c.abs().max(-1).values
            step = torch.pow(2.0, torch.ceil(torch.log2(top / 127)))
            step = torch.where(top > 127 * step, 2 * step, step)
            step = torch.where(top <= 63.5 * step, step / 2, step)[:, None]
            c = torch.round(c / step) * step
        r = turned(x[:, d_c:], pos)
        rows = torch.cat([c, r], -1)
        at = s["table"][b].long()[pos // page]
        pool[at, pos % page] = rows
        q_all.append(turned(s["q_rope"][t0:t0 + n], pos))
        t0 += n
    if case["op"] == "append" and case["cache"] == "native":
        return {"pool": pool, "q": torch.cat(q_all)}
    rows = torch.cat([pool[s["table"][b].long()].reshape(-1, d_c + d_r)[:s["total"][b]]
                      for b in range(case["batch"])])
    return {"rows": rows, "q": torch.cat(q_all)} if case["op"] == "append" else {"rows": rows}
