"""Cases of the attention operators: append to the paged cache, decode attention, prefill attention.

Every case has a plain form (elementary torch operations, 32-bit arithmetic, one rounding at the
end) and the framework's own call; `own` picks between them. Shapes are those of a decoder layer
around the MoE FFN of this repository: d = 7168 is 56 query heads of 128 (8 key heads: groups of
7), token batches are the batches of its sweep (1 .. 16384), and the rest are generic head
layouts (32 over 8, 64 over 8, 16 over 2 with heads of 64).
"""
import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-6


# ---- cases -----------------------------------------------------------------------------------

def _append(name, **kw):
    c = {"name": name, "op": "append", "B": 1, "Hq": 32, "Hkv": 8, "D": 128, "kv": "bf16",
         "page": 16, "new_min": 1, "new_max": 1, "ctx_min": 0, "ctx_max": 0, "rot": 128,
         "pairs": False, "norm": True}
    c.update(kw)
    return c


def _decode(name, **kw):
    c = {"name": name, "op": "decode", "B": 1, "Hq": 32, "Hkv": 8, "D": 128, "kv": "bf16",
         "page": 16, "len_min": 1, "len_max": 1, "window": 0, "sink": 0}
    c.update(kw)
    return c


def _prefill(name, **kw):
    c = {"name": name, "op": "prefill", "B": 1, "Hq": 32, "Hkv": 8, "D": 128, "kv": "bf16",
         "page": 16, "new_min": 1, "new_max": 1, "ctx_min": 0, "ctx_max": 0, "window": 0,
         "sink": 0}
    c.update(kw)
    return c


def listed():
    return [
        # one user's next token: nothing but latency
        _append("append_one", ctx_min=777, ctx_max=777),
        # a decode batch of 256 (the repository's headline batch) into an E4M3 cache
        _append("append_decode256_fp8", B=256, Hq=56, kv="fp8", ctx_min=1, ctx_max=640),
        # a step that admits a few prompts of odd lengths, 16384 tokens at most (the sweep's
        # largest batch); part of each head rotated, neighbouring pairs, larger pages
        _append("append_prompts", B=9, Hq=64, page=64, new_min=311, new_max=3001, rot=64,
                pairs=True),
        # one user's next token over a short chat
        _decode("decode_one", len_min=1003, len_max=1003),
        # an ordinary ragged batch, E4M3 cache, groups of 7 query heads
        _decode("decode_ragged_fp8", B=64, Hq=56, kv="fp8", len_min=1, len_max=4099),
        # one user over a very long document
        _decode("decode_long", Hq=64, page=64, len_min=131071, len_max=131071),
        # a full decode batch of long chats: the largest read of the cache
        _decode("decode_batch256", B=256, Hq=64, page=32, len_min=2048, len_max=8192),
        # window of 1024 with 4 first tokens that stay, small heads
        _decode("decode_window", B=96, Hq=16, Hkv=2, D=64, len_min=500, len_max=20000,
                window=1024, sink=4),
        # a short prompt on its own: latency
        _prefill("prefill_short", new_min=37, new_max=37),
        # a step of ragged prompts, groups of 7
        _prefill("prefill_ragged", B=8, Hq=56, new_min=65, new_max=3001),
        # one long prompt with a window of 1024 and 4 sinks
        _prefill("prefill_window", Hq=32, D=64, page=32, new_min=8192, new_max=8192, window=1024,
                 sink=4),
        # a chunk of 2048 tokens of a long document, over what is cached already in E4M3
        _prefill("prefill_chunk_fp8", Hq=64, kv="fp8", page=64, new_min=2048, new_max=2048,
                 ctx_min=20011, ctx_max=20011),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(["append", "decode", "prefill"])
        D = rng.choice([64, 128, 128])
        Hkv = rng.choice([1, 2, 4, 8, 8])
        c = {"op": op, "Hkv": Hkv, "Hq": Hkv * rng.choice([1, 2, 4, 7, 8, 16]), "D": D,
             "kv": rng.choice(["bf16", "bf16", "fp8"]), "page": rng.choice([8, 16, 16, 32, 64, 100, 128]),
             "B": _logint(rng, 1, 256)}
        if op == "decode":
            hi = _logint(rng, 1, 131072)
            c.update(len_min=_logint(rng, 1, hi), len_max=hi)
        else:
            new, ctx = _logint(rng, 1, 16384), rng.choice([0, _logint(rng, 1, 32768)])
            c.update(new_min=_logint(rng, 1, new), new_max=new,
                     ctx_min=_logint(rng, 1, ctx) if ctx else 0, ctx_max=ctx)
        if op == "append":
            c.update(rot=rng.choice([D, D, D // 2]), pairs=rng.random() < 0.5,
                     norm=rng.random() < 0.75)
        else:
            window = rng.choice([0, 0, _logint(rng, 16, 8192)])
            c.update(window=window, sink=rng.choice([0, 4, _logint(rng, 1, 200)]) if window else 0)
        lens, new = _lengths(c)
        w = work(c)
        if sum(new) > 16384 and op != "decode":
            continue
        # no more than the largest listed cases, and room for the plain form's whole score matrix
        if w["bytes"] > 5e9 or w["flops"] > 1.4e12 or sum(lens) * Hkv * D > 1.4e9:
            continue
        if c["B"] * c["Hq"] * max(new) * max(lens) > 4e9:
            continue
        if c["B"] * max(lens) * Hkv * D > 5e9:
            continue
        return c


def _lengths(case):
    """(cached keys, new tokens) of each sequence: spread evenly over their ranges, shuffled."""
    B = case["B"]
    rng = random.Random(B * 1000003 + case["D"])

    def spread(lo, hi):
        v = [lo + (hi - lo) * (i + 1) // B for i in range(B)]  # the last one is hi
        rng.shuffle(v)
        return v

    if case["op"] == "decode":
        return spread(case["len_min"], case["len_max"]), [1] * B
    new = spread(case["new_min"], case["new_max"])
    ctx = spread(case["ctx_min"], case["ctx_max"])
    return [a + b for a, b in zip(new, ctx)], new


def _visible(L, window, sink):
    """Keys that the token at position L - 1 sees."""
    return L if not window else min(L, window + min(sink, max(L - window, 0)))


def work(case):
    lens, new = _lengths(case)
    T, D, Hq, Hkv = sum(new), case["D"], case["Hq"], case["Hkv"]
    cb = 2 if case["kv"] == "bf16" else 1
    if case["op"] == "append":
        rows = min(T, max(lens))  # distinct positions, at most
        return {"bytes": T * (Hq + 2 * Hkv) * D * 2 + T * Hq * D * 2 + 2 * T * Hkv * D * cb
                + rows * case["rot"] * 4,
                "flops": T * (Hq + Hkv) * D * 8}
    W, S = case["window"], case["sink"]
    if case["op"] == "decode":
        keys = pairs = sum(_visible(L, W, S) for L in lens)
    else:
        keys = pairs = 0
        for L, n in zip(lens, new):
            pairs += sum(_visible(p + 1, W, S) for p in range(L - n, L))
            keys += min(L, (n + W - 1) + min(S, max(L - n - W + 1, 0))) if W else L
    return {"bytes": 2 * keys * Hkv * D * cb + 2 * T * Hq * D * 2 + T * Hq * 4,
            "flops": 4 * D * Hq * pairs}


# ---- inputs ----------------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    lens, new = _lengths(case)
    B, D, Hq, Hkv, page = case["B"], case["D"], case["Hq"], case["Hkv"], case["page"]
    T, fp8 = sum(new), case["kv"] == "fp8"
    pages = [-(-L // page) for L in lens]
    num_pages = sum(pages) + 3

    def normal(*size):
        return torch.randn(*size, generator=g, device=DEV, dtype=torch.bfloat16)

    def cache(scale):
        x = torch.empty(num_pages, Hkv, page, D, device=DEV, dtype=torch.bfloat16)
        x.normal_(generator=g)
        if fp8:
            for i in range(0, num_pages, 4096):
                x[i:i + 4096] /= scale[:, None, None]
            return x.to(torch.float8_e4m3fn)
        return x

    k_scale = v_scale = None
    if fp8:  # a calibrated scale for each key head: about 6 standard deviations to the largest code
        k_scale = torch.rand(Hkv, generator=g, device=DEV) * 0.01 + 0.01
        v_scale = torch.rand(Hkv, generator=g, device=DEV) * 0.01 + 0.01
    st = {"case": dict(case), "lens": lens, "new": new, "k_scale": k_scale, "v_scale": v_scale}
    st["k_cache"], st["v_cache"] = cache(k_scale), cache(v_scale)
    # the pages of a sequence lie anywhere in the cache; unused entries of the table are -1
    perm = torch.randperm(num_pages, generator=g, device=DEV).to(torch.int32)
    first = torch.tensor([0] + pages, device=DEV).cumsum(0)[:-1]
    col = torch.arange(max(pages), device=DEV)
    used = col[None, :] < torch.tensor(pages, device=DEV)[:, None]
    at = torch.where(used, first[:, None] + col[None, :], 0)
    st["block_table"] = torch.where(used, perm[at], -1).to(torch.int32).contiguous()
    st["kv_len"] = torch.tensor(lens, device=DEV, dtype=torch.int32)
    st["q_start"] = torch.tensor([0] + new, device=DEV).cumsum(0).to(torch.int32)
    if case["op"] == "append":
        st["qkv"] = normal(T, (Hq + 2 * Hkv) * D)  # the projection's output, one row a token
        st["q_out"] = torch.empty(T, Hq, D, device=DEV, dtype=torch.bfloat16)
        st["q_norm"] = st["k_norm"] = None
        if case["norm"]:
            st["q_norm"] = (1 + 0.1 * normal(D)).to(torch.bfloat16)
            st["k_norm"] = (1 + 0.1 * normal(D)).to(torch.bfloat16)
        half = case["rot"] // 2
        freq = 10000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)
        ang = torch.arange(max(lens), device=DEV, dtype=torch.float64)[:, None] * freq[None, :]
        st["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).to(torch.float32).contiguous()
    else:
        st["q"] = normal(T, Hq, D)
        st["o"] = torch.empty(T, Hq, D, device=DEV, dtype=torch.bfloat16)
        st["lse"] = torch.empty(T, Hq, device=DEV, dtype=torch.float32)
    if own:
        import routed_expert_ffn_moe_gb300 as moe

        more = {}
        if case["op"] == "append":
            row = (Hq + 2 * Hkv) * D
            more = dict(q_stride=row, k_stride=row, v_stride=row, rot_dim=case["rot"],
                        rot_pairs=case["pairs"], max_pos=max(lens), eps=EPS)
        else:
            more = dict(window=case["window"], n_sink=case["sink"])
        st["shape"] = moe.attn_shape(T=T, B=B, Hq=Hq, Hkv=Hkv, D=D, kv_dtype=case["kv"],
                                     page_size=page, max_pages=st["block_table"].shape[1],
                                     num_pages=num_pages, **more)
        st["ws"] = torch.zeros(moe.moe_attn_workspace_size(st["shape"], case["op"] == "prefill"),
                               dtype=torch.uint8, device=DEV)
    return st


# ---- one pass --------------------------------------------------------------------------------

def run(st):
    op = st["case"]["op"]
    if own:
        return _run_own(st, op)
    return {"append": _plain_append, "decode": _plain_decode, "prefill": _plain_prefill}[op](st)


def _run_own(st, op):
    import routed_expert_ffn_moe_gb300 as moe

    s = st["shape"]
    if op == "append":
        c = st["case"]
        nq, nk = c["Hq"] * c["D"], c["Hkv"] * c["D"]
        qkv = st["qkv"]
        moe.moe_attn_append(s, qkv[:, :nq], qkv[:, nq:nq + nk], qkv[:, nq + nk:], st["q_norm"],
                            st["k_norm"], st["cos_sin"], None, st["block_table"], st["kv_len"],
                            st["q_start"], st["k_scale"], st["v_scale"], st["q_out"],
                            st["k_cache"], st["v_cache"], st["ws"])
        return {"q": st["q_out"], "k": st["k_cache"], "v": st["v_cache"]}
    if op == "decode":
        moe.moe_attn_decode(s, st["q"], st["k_cache"], st["v_cache"], st["k_scale"],
                            st["v_scale"], st["block_table"], st["kv_len"], st["o"], st["lse"],
                            st["ws"])
    else:
        moe.moe_attn_prefill(s, st["q"], st["k_cache"], st["v_cache"], st["k_scale"],
                             st["v_scale"], st["block_table"], st["kv_len"], st["q_start"],
                             st["o"], st["lse"], st["ws"])
    return {"o": st["o"], "lse": st["lse"]}


def _token_places(st):
    """Of each new token: its sequence, its number among the new ones, its place in the cache."""
    t = torch.arange(sum(st["new"]), device=DEV)
    start = st["q_start"].long()
    b = (t[:, None] >= start[None, 1:]).sum(1)
    i = t - start[b]
    n = start[b + 1] - start[b]
    return b, i, st["kv_len"].long()[b] - n + i


def _plain_append(st):
    c = st["case"]
    D, Hq, Hkv, half = c["D"], c["Hq"], c["Hkv"], c["rot"] // 2
    x = st["qkv"].float().view(-1, Hq + 2 * Hkv, D)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    b, _, pos = _token_places(st)
    cos, sin = st["cos_sin"][pos, None, :half], st["cos_sin"][pos, None, half:]

    def turned(y, w):
        if w is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w.float()
        if c["pairs"]:
            a, e = y[..., 0:2 * half:2], y[..., 1:2 * half:2]
            r = torch.stack([a * cos - e * sin, e * cos + a * sin], -1).flatten(-2)
        else:
            a, e = y[..., :half], y[..., half:2 * half]
            r = torch.cat([a * cos - e * sin, e * cos + a * sin], -1)
        return torch.cat([r, y[..., 2 * half:]], -1)

    q, k = turned(q, st["q_norm"]), turned(k, st["k_norm"])
    at = st["block_table"][b, pos // c["page"]].long()
    off = pos % c["page"]
    if c["kv"] == "fp8":
        k = (k / st["k_scale"][:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        v = (v / st["v_scale"][:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        st["k_cache"].view(torch.uint8)[at, :, off] = k.view(torch.uint8)
        st["v_cache"].view(torch.uint8)[at, :, off] = v.view(torch.uint8)
    else:
        st["k_cache"][at, :, off] = k.to(torch.bfloat16)
        st["v_cache"][at, :, off] = v.to(torch.bfloat16)
    return {"q": q.to(torch.bfloat16), "k": st["k_cache"], "v": st["v_cache"]}


def _cached(x, scale, table):
    """A cache's rows of every sequence, in 32 bits: [B, Hkv, longest, D]."""
    x = x[table.clamp(min=0).long()].float()          # [B, pages, Hkv, page, D]
    x = x.permute(0, 2, 1, 3, 4).flatten(2, 3)
    return x if scale is None else x * scale[:, None, None]


def _softmax_product(s, seen, v):
    """softmax over the seen keys times v, and the logarithm of the sum; zeros where none is."""
    s = torch.where(seen, s, -math.inf)
    m = s.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(total > 0, total, 1.0)
    return o, (m + torch.log(total)).squeeze(-1)


def _seen(j, pos, window, sink):
    ok = (j <= pos) & (pos >= 0)
    return ok & ((pos - j < window) | (j < sink)) if window else ok


def _plain_decode(st):
    c = st["case"]
    B, D, Hq, Hkv = c["B"], c["D"], c["Hq"], c["Hkv"]
    k = _cached(st["k_cache"], st["k_scale"], st["block_table"])
    q = st["q"].float().view(B, Hkv, Hq // Hkv, D)
    s = (q @ k.transpose(-1, -2)) * (1.0 / math.sqrt(D))
    del k
    j = torch.arange(s.shape[-1], device=DEV)
    seen = _seen(j, (st["kv_len"].long() - 1)[:, None, None, None], c["window"], c["sink"])
    o, lse = _softmax_product(s, seen, _cached(st["v_cache"], st["v_scale"], st["block_table"]))
    return {"o": o.reshape(B, Hq, D).to(torch.bfloat16), "lse": lse.reshape(B, Hq)}


def _plain_prefill(st):
    c = st["case"]
    B, D, Hq, Hkv = c["B"], c["D"], c["Hq"], c["Hkv"]
    G, n = Hq // Hkv, max(st["new"])
    k = _cached(st["k_cache"], st["k_scale"], st["block_table"])
    b, i, _ = _token_places(st)
    q = torch.zeros(B, n, Hq, D, device=DEV)
    q[b, i] = st["q"].float()
    q = q.view(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    s = ((q @ k.transpose(-1, -2)) * (1.0 / math.sqrt(D))).view(B, Hkv, G, n, -1)
    del k
    new = (st["q_start"][1:] - st["q_start"][:-1]).long()
    pos = (st["kv_len"].long() - new)[:, None] + torch.arange(n, device=DEV)[None, :]
    j = torch.arange(s.shape[-1], device=DEV)
    seen = _seen(j, pos[:, None, None, :, None], c["window"], c["sink"])
    v = _cached(st["v_cache"], st["v_scale"], st["block_table"])[:, :, None]
    o, lse = _softmax_product(s, seen, v)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D)[b, i]
    lse = lse.permute(0, 3, 1, 2).reshape(B, n, Hq)[b, i]
    return {"o": o.to(torch.bfloat16), "lse": lse}


# ---- the definition in 64 bits ---------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    f64 = torch.float64
    D, Hq, Hkv, page = case["D"], case["Hq"], case["Hkv"], case["page"]
    G, table = Hq // Hkv, st["block_table"].cpu()
    if case["op"] == "append":
        kc, vc = st["k_cache"].to(f64), st["v_cache"].to(f64)
        qo = torch.empty(sum(st["new"]), Hq, D, device=DEV, dtype=f64)
        R = case["rot"]
        lo, hi = (slice(0, R, 2), slice(1, R, 2)) if case["pairs"] else (slice(0, R // 2),
                                                                          slice(R // 2, R))
        ks = st["k_scale"].to(f64)[None, :, None] if st["k_scale"] is not None else 1.0
        vs = st["v_scale"].to(f64)[None, :, None] if st["v_scale"] is not None else 1.0
        t0 = 0
        for b, (L, n) in enumerate(zip(st["lens"], st["new"])):
            rows = st["qkv"][t0:t0 + n].to(f64).view(n, -1, D)
            cs = st["cos_sin"][L - n:L].to(f64)[:, None]
            outs = []
            for x, w in ((rows[:, :Hq], st["q_norm"]), (rows[:, Hq:Hq + Hkv], st["k_norm"])):
                if w is not None:
                    x = w.to(f64) * x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / D + EPS)
                z = torch.view_as_complex(torch.stack([x[..., lo], x[..., hi]], -1).contiguous())
                z = z * torch.complex(cs[..., :R // 2].contiguous(), cs[..., R // 2:].contiguous())
                x = x.clone()
                x[..., lo], x[..., hi] = z.real, z.imag
                outs.append(x)
            qo[t0:t0 + n] = outs[0]
            p = torch.arange(L - n, L)
            where = table[b, p // page].long().to(DEV), (p % page).to(DEV)
            kc.permute(0, 2, 1, 3)[where] = outs[1] / ks
            vc.permute(0, 2, 1, 3)[where] = rows[:, Hq + Hkv:] / vs
            t0 += n
        if case["kv"] == "fp8":
            kc, vc = kc.clamp(-448, 448), vc.clamp(-448, 448)
        return {"q": qo, "k": kc, "v": vc}
    o = torch.zeros(sum(st["new"]), Hq, D, device=DEV, dtype=f64)
    lse = torch.full((sum(st["new"]), Hq), -math.inf, device=DEV, dtype=f64)
    W, S, t0 = case["window"], case["sink"], 0
    for b, (L, n) in enumerate(zip(st["lens"], st["new"])):
        ids = table[b, :-(-L // page)].long().to(DEV)
        for h in range(Hkv):
            k = st["k_cache"][ids, h].to(f64).reshape(-1, D)[:L]
            v = st["v_cache"][ids, h].to(f64).reshape(-1, D)[:L]
            if st["k_scale"] is not None:
                k, v = k * st["k_scale"][h].to(f64), v * st["v_scale"][h].to(f64)
            for i0 in range(0, n, 1024):
                i1 = min(n, i0 + 1024)
                q = st["q"][t0 + i0:t0 + i1, h * G:(h + 1) * G].to(f64)
                pos = torch.arange(L - n + i0, L - n + i1, device=DEV)[:, None, None]
                end = L - n + i1  # later keys are hidden from all of these
                s = torch.einsum("tgd,jd->tgj", q, k[:end]) / math.sqrt(D)
                j = torch.arange(end, device=DEV)[None, None, :]
                hidden = j > pos
                if W:
                    hidden |= (j + W <= pos) & (j >= S)
                s.masked_fill_(hidden, -math.inf)
                at = lse[t0 + i0:t0 + i1, h * G:(h + 1) * G]
                at.copy_(torch.logsumexp(s, -1))
                s.sub_(at[..., None]).exp_()
                o[t0 + i0:t0 + i1, h * G:(h + 1) * G] = torch.einsum("tgj,jd->tgd", s, v[:end])
        t0 += n
    return {"o": o, "lse": lse}
