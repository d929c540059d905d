"""Cases of the attention-side operators of a decoder layer: per-head norm and
rotation of queries and keys, the 4-bit key/value cache (written and read back),
and attention over that cache.

The cache is a uint8 tensor [pages][heads][2][64 * (D / 2 + 4)] (index 2: K, V).  A
page holds 64 tokens; a block is 64 rows of D / 2 code bytes (element 2 i in the low
four bits of byte i, 2 i + 1 in the high ones) followed by 64 bf16 pairs (step s, low
end m); an element stands for m + s * code.  Sequence b of a batch has ctx_lens[b] tokens,
position p in slot p % 64 of page page_table[b][p // 64].  The new tokens of a batch are
rows cu_q[b] .. cu_q[b + 1] of the ragged tensors and the last ones of their sequence;
without cu_q every sequence has one.
"""
import math
import random

import torch

own = False

PAGE = 64


def _framework():
    from bit_gemv_sherry_b200 import sherry
    return sherry


_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of one sequence of a 1B-shaped decoder: the fp32 outputs of its q
        # and k GEMVs, rotated into bf16; the smallest call, latency only
        dict(name="rope_decode_1", op="rope", tokens=1, hq=32, hk=8, dim=64, rot=64, src="f32",
             dst="bf16", norm=False, pairs=False, far=8191),
        # prefill of 2048 tokens of the same decoder, from the GEMM's fp32 outputs
        dict(name="rope_prefill_2048", op="rope", tokens=2048, hq=32, hk=8, dim=64, rot=64,
             src="f32", dst="bf16", norm=False, pairs=False, far=2047),
        # a decoder with normed queries and keys, heads of 128, an odd number of tokens
        # far into a long context; adjacent pairs rotated, half of each head left alone
        dict(name="rope_norm_long", op="rope", tokens=8191, hq=32, hk=8, dim=128, rot=64,
             src="bf16", dst="bf16", norm=True, pairs=True, far=131071),
        # a decode step of 16 sequences written to the cache and read back
        dict(name="cache_decode_16", op="cache", seqs=16, new=1, ctx=4096, heads=8, dim=64,
             src="f32", dst="f32", ragged=3),
        # prefill of a ragged batch, 1B-shaped, values from the fp32 GEMM outputs
        dict(name="cache_prefill_ragged", op="cache", seqs=5, new=1000, ctx=3000, heads=8, dim=64,
             src="f32", dst="bf16", ragged=11),
        # a long prompt in bf16, heads of 128
        dict(name="cache_prompt_32k", op="cache", seqs=1, new=32768, ctx=32768, heads=8, dim=128,
             src="bf16", dst="bf16", ragged=0),
        # one sequence decoding: latency
        dict(name="attn_decode_1x2k", op="attn", seqs=1, new=1, ctx=2048, hq=32, hk=8, dim=64,
             ragged=0),
        # a served batch of odd lengths, an empty slot among them
        dict(name="attn_decode_16_ragged", op="attn", seqs=16, new=1, ctx=8192, hq=32, hk=8, dim=64,
             ragged=5),
        # many long sequences, heads of 128: the cache's bandwidth
        dict(name="attn_decode_32x32k", op="attn", seqs=32, new=1, ctx=32768, hq=32, hk=8, dim=128,
             ragged=0),
        # a few drafted tokens per sequence checked at once
        dict(name="attn_drafts_7", op="attn", seqs=7, new=5, ctx=5001, hq=12, hk=4, dim=128,
             ragged=9),
        # prefill of one 2048-token prompt, 1B-shaped
        dict(name="attn_prefill_2048", op="attn", seqs=1, new=2048, ctx=2048, hq=32, hk=8, dim=64,
             ragged=0),
        # the next 4096 tokens of long prompts, heads of 128: tensor cores
        dict(name="attn_chunk_4x16k", op="attn", seqs=4, new=4096, ctx=16384, hq=32, hk=8, dim=128,
             ragged=0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_one(rng, op):
    dim = rng.choice([64, 128])
    if op == "rope":
        hk = rng.choice([1, 2, 4, 8])
        return dict(op=op, tokens=_log_int(rng, 1, 8191), hq=hk * rng.choice([1, 2, 3, 4, 7, 8]), hk=hk,
                    dim=dim, rot=rng.choice([dim, dim, dim // 2]), src=rng.choice(["f32", "bf16"]),
                    dst=rng.choice(["f32", "bf16"]), norm=rng.random() < 0.5,
                    pairs=rng.random() < 0.5, far=_log_int(rng, 1, 131071))
    if op == "cache":
        new = 1 if rng.random() < 0.3 else _log_int(rng, 2, 32768)
        return dict(op=op, seqs=_log_int(rng, 1, 64), new=new, ctx=_log_int(rng, new, 65536),
                    heads=rng.choice([1, 2, 4, 8]), dim=dim, src=rng.choice(["f32", "bf16"]),
                    dst=rng.choice(["f32", "bf16"]), ragged=rng.choice([0, rng.randrange(1, 10 ** 6)]))
    hk = rng.choice([1, 2, 4, 8])
    kind = rng.random()
    new = 1 if kind < 0.45 else rng.randint(2, 16) if kind < 0.6 else _log_int(rng, 17, 4096)
    return dict(op=op, seqs=_log_int(rng, 1, 64), new=new, ctx=_log_int(rng, new, 32768),
                hq=hk * rng.choice([1, 2, 3, 4, 6, 8]), hk=hk, dim=dim,
                ragged=rng.choice([0, rng.randrange(1, 10 ** 6)]))


def draw(rng):
    op = rng.choice(["rope", "cache", "attn", "attn"])
    most = [work(c) for c in listed() if c["op"] == op]
    top = {k: max(w[k] for w in most) for k in ("bytes", "flops")}
    while True:
        case = _draw_one(rng, op)
        w = work(case)
        if w["bytes"] <= top["bytes"] and w["flops"] <= top["flops"]:
            return case


def _lens(case):
    """(context lengths, new tokens) of a case's sequences: all the same, or drawn from
    the case's own number, with an empty slot in batches of four and more."""
    n = case["seqs"]
    if not case["ragged"]:
        return [case["ctx"]] * n, [case["new"]] * n
    r = random.Random(case["ragged"])
    ctx = [r.randint(1, case["ctx"]) for _ in range(n)]
    ctx[r.randrange(n)] = case["ctx"]
    new = [min(c, case["new"] if case["new"] == 1 else r.randint(1, case["new"])) for c in ctx]
    if n >= 4:
        i = r.randrange(n)
        ctx[i], new[i] = 0, 1
    return ctx, new


def work(case):
    if case["op"] == "rope":
        rows = case["tokens"] * (case["hq"] + case["hk"])
        size = 4 if case["src"] == "f32" else 2
        out = 4 if case["dst"] == "f32" else 2
        return {"bytes": rows * case["dim"] * (size + out) + 4 * case["tokens"],
                "flops": rows * (3 * case["rot"] + (4 * case["dim"] if case["norm"] else 0))}
    ctx, new = _lens(case)
    dim = case["dim"]
    if case["op"] == "cache":
        # two tensors (K and V) read, coded into the cache, read from it, written out
        rows = 2 * sum(min(c, n) for c, n in zip(ctx, new)) * case["heads"]
        size = 4 if case["src"] == "f32" else 2
        out = 4 if case["dst"] == "f32" else 2
        return {"bytes": rows * (dim * (size + out) + 2 * (dim // 2 + 4)), "flops": rows * 6 * dim}
    pairs = sum(n * c - n * (n - 1) // 2 for c, n in zip(ctx, new) if c)
    return {"bytes": sum(ctx) * case["hk"] * 2 * (dim // 2 + 4) + 4 * sum(new) * case["hq"] * dim,
            "flops": 4 * dim * case["hq"] * pairs}


# ----------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _keys(shape, g):
    """Keys as a decoder makes them: a few channels much larger than the others, off centre."""
    x = torch.randn(shape, generator=g, device="cuda")
    ch = torch.randn(shape[-2:], generator=g, device="cuda")
    return x * 0.8 + torch.where(ch > 1.8, 3.0 * ch, 0.3 * ch)


def _batch(case, seed):
    """Lengths, page table (pages in no order, a few to spare) and the offsets of the rows."""
    ctx, new = _lens(case)
    need = [(c + PAGE - 1) // PAGE for c in ctx]
    width = max(max(need), 1)
    pages = sum(need) + 3
    g = torch.Generator()
    g.manual_seed(seed)
    order = torch.randperm(pages, generator=g)
    table = torch.zeros(len(ctx), width, dtype=torch.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    one = all(n == 1 for n in new)
    return dict(ctx=ctx, new=new, cu=cu, pages=pages, tokens=cu[-1], max_q=max(new),
                table=table.cuda(), lens=torch.tensor(ctx, dtype=torch.int32).cuda(),
                cu_q=None if one else torch.tensor(cu, dtype=torch.int32).cuda())


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "rope":
        t, dim, rot = case["tokens"], case["dim"], case["rot"]
        src, dst = _DTYPES[case["src"]], _DTYPES[case["dst"]]
        st = dict(op="rope", pairs=case["pairs"], eps=1e-5,
                  q=torch.randn(t, case["hq"], dim, generator=g, device="cuda").to(src),
                  k=_keys((t, case["hk"], dim), g).to(src),
                  inv_freq=(500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda(),
                  qw=None, kw=None)
        start = case["far"] - (t - 1)
        if start >= 0:  # one sequence's consecutive tokens, the last at `far`
            st["pos"] = torch.arange(start, case["far"] + 1, dtype=torch.int32, device="cuda")
        else:           # a batch of short sequences
            st["pos"] = torch.randint(0, case["far"] + 1, (t,), generator=g, device="cuda").int()
        if case["norm"]:
            st["qw"] = 1.0 + 0.2 * torch.randn(dim, generator=g, device="cuda")
            st["kw"] = 1.0 + 0.2 * torch.randn(dim, generator=g, device="cuda")
        st["q_out"] = torch.empty(st["q"].shape, dtype=dst, device="cuda")
        st["k_out"] = torch.empty(st["k"].shape, dtype=dst, device="cuda")
        return st
    st = dict(_batch(case, seed), op=case["op"], dim=case["dim"])
    dim = case["dim"]
    if case["op"] == "cache":
        src = _DTYPES[case["src"]]
        shape = (st["tokens"], case["heads"], dim)
        st["k"] = _keys(shape, g).to(src)
        st["v"] = torch.randn(shape, generator=g, device="cuda").to(src)
        st["cache"] = torch.zeros(st["pages"], case["heads"], 2, PAGE * (dim // 2 + 4), dtype=torch.uint8,
                                  device="cuda")
        dst = _DTYPES[case["dst"]]
        # rows without a slot (an empty sequence's) are not read back: they stay zero
        st["k_out"] = torch.zeros(shape, dtype=dst, device="cuda")
        st["v_out"] = torch.zeros(shape, dtype=dst, device="cuda")
        return st
    # a cache of keys and values as earlier steps left it
    st["scale"] = 1.0 / math.sqrt(dim)
    st["q"] = torch.randn(st["tokens"], case["hq"], dim, generator=g, device="cuda").bfloat16()
    cache = torch.empty(st["pages"], case["hk"], 2, PAGE * (dim // 2 + 4), dtype=torch.uint8, device="cuda")
    ch = torch.randn(case["hk"], 1, dim, generator=g, device="cuda")
    off = torch.where(ch > 1.8, 3.0 * ch, 0.3 * ch)
    step = max(1, (1 << 26) // (case["hk"] * PAGE * dim))
    for a in range(0, st["pages"], step):
        n = min(step, st["pages"] - a)
        for i in range(2):
            x = torch.randn(n, case["hk"], PAGE, dim, generator=g, device="cuda")
            codes, s, m = _quantize(x * 0.8 + off if i == 0 else x)
            blk = cache[a:a + n, :, i]
            blk[..., :PAGE * dim // 2] = _to_bytes(codes).flatten(-2)
            blk[..., PAGE * dim // 2:] = torch.stack([s, m], -1).flatten(-2).view(torch.uint8)
    st["cache"] = cache
    st["out"] = torch.empty(st["tokens"], case["hq"], dim, dtype=torch.bfloat16, device="cuda")
    return st


# ----------------------------------------------------------------------------- plain form
def _quantize(x):
    """Codes, step and low end of the last axis: the cache's definition, in 32 bits."""
    lo, hi = x.amin(-1), x.amax(-1)
    s = ((hi - lo) * torch.tensor(1.0 / 15.0, dtype=torch.float32, device=x.device)).bfloat16()
    m = lo.bfloat16()
    sf = s.float()
    inv = torch.where(sf > 0, torch.ones_like(sf) / sf, torch.zeros_like(sf))
    codes = torch.round((x - m.float().unsqueeze(-1)) * inv.unsqueeze(-1)).clamp(0, 15)
    return codes, s, m


def _to_bytes(codes):
    c = codes.to(torch.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4)


def _values(blk, dim):
    """The fp32 values of blocks [..., 64 * (D / 2 + 4)] -> [..., 64, D]."""
    n = PAGE * dim // 2
    codes = blk[..., :n].unflatten(-1, (PAGE, dim // 2))
    sm = blk[..., n:].contiguous().view(torch.bfloat16).unflatten(-1, (PAGE, 2)).float()
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
    return sm[..., 1:] + sm[..., :1] * c


def _rope_one(x, w, st):
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + st["eps"]) * w
    ang = st["pos"].double()[:, None] * st["inv_freq"].double()
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]
    half = st["inv_freq"].numel()
    out = y.clone()
    if st["pairs"]:
        a, b = y[..., 0:2 * half:2], y[..., 1:2 * half:2]
        out[..., 0:2 * half:2], out[..., 1:2 * half:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = y[..., :half], y[..., half:2 * half]
        out[..., :half], out[..., half:2 * half] = a * cos - b * sin, b * cos + a * sin
    return out


def _slots(st):
    """Row, page and slot of every new token that has one."""
    rows, pos, seq = [], [], []
    for b, (c, n) in enumerate(zip(st["ctx"], st["new"])):
        k = min(c, n)
        rows.append(torch.arange(st["cu"][b] + n - k, st["cu"][b] + n))
        pos.append(torch.arange(c - k, c))
        seq.append(torch.full((k,), b))
    rows, pos, seq = (torch.cat(a).cuda() for a in (rows, pos, seq))
    return rows, st["table"][seq, pos // PAGE].long(), pos % PAGE


def _run_plain(st):
    if st["op"] == "rope":
        st["q_out"].copy_(_rope_one(st["q"], st["qw"], st))
        st["k_out"].copy_(_rope_one(st["k"], st["kw"], st))
        return st["q_out"], st["k_out"]
    dim = st["dim"]
    if st["op"] == "cache":
        rows, page, slot = _slots(st)
        cache = st["cache"]
        n = PAGE * dim // 2
        codes_at = cache[..., :n].unflatten(-1, (PAGE, dim // 2))
        sm_at = cache[..., n:].unflatten(-1, (PAGE, 4))
        for i, (x, out) in enumerate(((st["k"], st["k_out"]), (st["v"], st["v_out"]))):
            codes, s, m = _quantize(x[rows].float())
            codes_at[page, :, i, slot] = _to_bytes(codes)
            sm_at[page, :, i, slot] = torch.stack([s, m], -1).view(torch.uint8)
            b = codes_at[page, :, i, slot]
            sm = sm_at[page, :, i, slot].contiguous().view(torch.bfloat16).float()
            c = torch.stack([b & 15, b >> 4], -1).flatten(-2).float()
            out[rows] = (sm[..., 1:] + sm[..., :1] * c).to(out.dtype)
        return st["k_out"], st["v_out"]
    out = st["out"]
    hq = st["q"].shape[1]
    hk = st["cache"].shape[1]
    grp = hq // hk
    for b, (c, n) in enumerate(zip(st["ctx"], st["new"])):
        r0 = st["cu"][b]
        if c == 0:
            out[r0:r0 + n] = 0
            continue
        blk = st["cache"][st["table"][b, :(c + PAGE - 1) // PAGE].long()]
        q = st["q"][r0:r0 + n].float().unflatten(1, (hk, grp))
        seen = torch.arange(c, device="cuda")[None, :] <= torch.arange(c - n, c, device="cuda")[:, None]
        per = max(1, min(hk, (1 << 28) // (n * grp * c)))
        for h in range(0, hk, per):
            k = _values(blk[:, h:h + per, 0], dim).transpose(0, 1).flatten(1, 2)[:, :c]
            v = _values(blk[:, h:h + per, 1], dim).transpose(0, 1).flatten(1, 2)[:, :c]
            qh = q[:, h:h + per].permute(1, 2, 0, 3)                       # head, group, token, D
            s = torch.matmul(qh, k[:, None].transpose(-1, -2)) * st["scale"]
            s = s.masked_fill(~seen, float("-inf"))
            p = torch.exp(s - s.amax(-1, keepdim=True))
            o = torch.matmul(p, v[:, None]) / p.sum(-1, keepdim=True)
            out[r0:r0 + n].unflatten(1, (hk, grp))[:, h:h + per] = o.permute(2, 0, 1, 3).to(out.dtype)
    return out


# ----------------------------------------------------------------------------- the framework's calls
def _run_own(st):
    S = _framework()
    if st["op"] == "rope":
        return S.qk_norm_rope(st["q"], st["k"], st["pos"], st["inv_freq"], q_weight=st["qw"], k_weight=st["kw"],
                              eps=st["eps"], interleaved=st["pairs"], q_out=st["q_out"], k_out=st["k_out"])
    if st["op"] == "cache":
        S.kv4_write(st["cache"], st["k"], st["v"], st["table"], st["lens"], cu_q=st["cu_q"])
        return S.kv4_read(st["cache"], st["table"], st["lens"], cu_q=st["cu_q"], k=st["k_out"], v=st["v_out"])
    return S.attn_kv4(st["q"], st["cache"], st["table"], st["lens"], cu_q=st["cu_q"], max_q=st["max_q"],
                      scale=st["scale"], out=st["out"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ----------------------------------------------------------------------------- the definition in 64 bits
def _exact_rope(x, w, st):
    y = x.double()
    if w is not None:
        y = y / ((y ** 2).sum(-1, keepdim=True) / y.shape[-1] + st["eps"]).sqrt() * w.double()
    r = st["inv_freq"].numel()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       torch.outer(st["pos"].double(), st["inv_freq"].double()))[:, None, :]
    head, rest = y[..., :2 * r], y[..., 2 * r:]
    if st["pairs"]:
        z = torch.view_as_real(torch.view_as_complex(head.unflatten(-1, (r, 2)).contiguous()) * turn).flatten(-2)
    else:
        z = torch.complex(head[..., :r].contiguous(), head[..., r:].contiguous()) * turn
        z = torch.cat([z.real, z.imag], -1)
    return torch.cat([z, rest], -1)


def _exact_cache(x, shape, st):
    """Rows as the cache holds them.  The definition rounds the step, the low end, the
    difference, the reciprocal and their product to 32 bits (the step and the low end to
    bf16 after that); 64-bit operations followed by those roundings give the same codes."""
    def f32(t):
        return t.to(torch.float32).double()

    def bf16(t):
        return t.to(torch.float32).to(torch.bfloat16).double()

    out = torch.zeros(shape, dtype=torch.float64, device="cuda")
    third = f32(torch.tensor(1.0 / 15.0, dtype=torch.float64, device="cuda"))
    for b, (c, n) in enumerate(zip(st["ctx"], st["new"])):
        k = min(c, n)
        r = slice(st["cu"][b] + n - k, st["cu"][b] + n)
        y = x[r].double()
        if y.numel() == 0:
            continue
        m = y.min(-1, keepdim=True).values
        s = bf16(f32(f32(y.max(-1, keepdim=True).values - m) * third))
        m = bf16(m)
        inv = torch.where(s > 0, f32(1.0 / s), torch.zeros_like(s))
        out[r] = m + s * f32(f32(y - m) * inv).round().clamp(0, 15)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(st["q"], st["qw"], st), _exact_rope(st["k"], st["kw"], st)
    if case["op"] == "cache":
        return _exact_cache(st["k"], st["k_out"].shape, st), _exact_cache(st["v"], st["v_out"].shape, st)
    dim, hk = case["dim"], case["hk"]
    grp = case["hq"] // hk
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    nib = torch.arange(256, device="cuda")
    pair = torch.stack([nib % 16, nib // 16], -1).double()                 # byte -> its two codes
    for b, (c, n) in enumerate(zip(st["ctx"], st["new"])):
        if c == 0:
            continue
        pages = st["table"][b].long()[torch.arange(c, device="cuda") // PAGE]
        slot = torch.arange(c, device="cuda") % PAGE
        last = torch.arange(n, device="cuda") + (c - n)
        for h in range(hk):
            kv = []
            for i in range(2):
                blk = st["cache"][:, h, i]
                rows = blk[:, :PAGE * dim // 2].reshape(-1, PAGE, dim // 2)[pages, slot].long()
                sm = blk[:, PAGE * dim // 2:].reshape(-1, PAGE, 4).view(torch.bfloat16)[pages, slot].double()
                kv.append(sm[:, 1:2] + sm[:, 0:1] * pair[rows].reshape(c, dim))
            for j in range(h * grp, (h + 1) * grp):
                e = st["q"][st["cu"][b]:st["cu"][b] + n, j].double() @ kv[0].T * st["scale"]
                e[torch.arange(c, device="cuda")[None] > last[:, None]] = -math.inf
                out[st["cu"][b]:st["cu"][b] + n, j] = torch.softmax(e, -1) @ kv[1]
    return out
