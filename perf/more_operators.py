"""Cases of the expert selection and the MXFP4 operators: scored and grouped routing from logits,
quantisation to MXFP4 and back, and the product of two MXFP4 matrices.

Every case has a plain form (elementary torch operations) and the framework's own call; `own` picks
between them. Sizes are those of this repository's layers: d = 7168, 256 and 384 routed experts, token
batches of its sweep (1 .. 16384), the attention's 56 + 8 + 8 heads of 128 as one projection of 9216
features; the rest are generic and odd ones.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ---- cases -----------------------------------------------------------------------------------

def _select(name, **kw):
    c = {"name": name, "op": "select", "T": 1, "E": 256, "k": 8, "score": "sigmoid", "bias": True,
         "groups": 1, "keep": 1, "group_top": 2, "renorm": True, "scale": 2.5}
    c.update(kw)
    return c


def _quant(name, **kw):
    c = {"name": name, "op": "quant", "rows": 1, "K": 7168, "dtype": "bf16", "pad": 0, "tiles": False}
    c.update(kw)
    return c


def _linear(name, **kw):
    c = {"name": name, "op": "linear", "T": 1, "K": 7168, "N": 7168, "x": "bf16", "bias": False,
         "residual": False}
    c.update(kw)
    return c


def listed():
    return [
        # one user's next token: nothing but latency
        _select("select_one", groups=8, keep=4),
        # a decode batch of the 384-expert layer, no groups
        _select("select_batch_384", T=256, E=384, k=6),
        # the largest prefill batch of the sweep, groups of experts
        _select("select_prompts", T=16384, groups=8, keep=4),
        # softmax scores, the best expert speaks for its group, weights as they are, an odd batch
        _select("select_softmax_odd", T=4099, E=160, k=6, score="softmax", bias=False, groups=8, keep=3,
                group_top=1, renorm=False, scale=16.0),
        # the activations of a decode batch, scales in the product's tiles
        _quant("quant_activations", rows=256, tiles=True),
        # gate and up weights of 8 experts, turned to 4 bits when a model is loaded
        _quant("quant_weights", rows=8 * 4096),
        # fp32 rows apart from each other, no size a power of two
        _quant("quant_fp32_odd", rows=777, K=2080, dtype="f32", pad=36),
        # one user's next token through the qkv projection: 34 MB of weights
        _linear("linear_one", N=9216),
        # a small decode batch through the output projection, the residual stream added
        _linear("linear_batch24", T=24, residual=True),
        # a decode batch whose activations are in 4 bits already
        _linear("linear_batch256", T=256, N=9216, x="mxfp4"),
        # odd sizes, a bias
        _linear("linear_odd", T=1003, K=2080, N=4099, bias=True),
        # the largest prefill batch through the qkv projection
        _linear("linear_prompts", T=16384, N=9216),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["select", "quant", "linear", "linear"])
    while True:
        if op == "select":
            groups = rng.choice([1, 1, 2, 4, 8, 8, 16])
            per = rng.choice([2, 4, 8, 16, 20, 24, 32, 33, 48, 64, 128])
            E = groups * per
            keep = rng.randint(1, groups)
            k = rng.choice([1, 2, 4, 6, 8, 8, 16])
            if E > 1024 or E < 4 or k > keep * per:
                continue
            return {"op": op, "T": _logint(rng, 1, 16384), "E": E, "k": k,
                    "score": rng.choice(["sigmoid", "softmax"]), "bias": rng.random() < 0.7,
                    "groups": groups, "keep": keep, "group_top": rng.choice([1, 2, 2]),
                    "renorm": rng.random() < 0.7, "scale": rng.choice([1.0, 2.5, 16.0])}
        K = 32 * _logint(rng, 1, 512)
        if op == "quant":
            rows = _logint(rng, 1, 65536)
            if rows * K > 8 * 4096 * 7168:
                continue
            return {"op": op, "rows": rows, "K": K, "dtype": rng.choice(["bf16", "bf16", "f32"]),
                    "pad": rng.choice([0, 0, 8 * rng.randint(1, 40)]), "tiles": rng.random() < 0.5}
        T, N = _logint(rng, 1, 16384), _logint(rng, 16, 20000)
        if rng.random() < 0.5:
            N = -(-N // 128) * 128
        if T * N * K > 16384 * 9216 * 7168 or N * K < 1 << 16:
            continue
        return {"op": op, "T": T, "K": K, "N": N, "x": rng.choice(["bf16", "bf16", "mxfp4"]),
                "bias": rng.random() < 0.4, "residual": rng.random() < 0.4}


def work(case):
    if case["op"] == "select":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": T * E * 4 + (E * 4 if case["bias"] else 0) + T * k * 8, "flops": T * E * 10}
    if case["op"] == "quant":  # there and back
        n = case["rows"] * case["K"]
        return {"bytes": n * (2 if case["dtype"] == "bf16" else 4) * 2 + n * 17 // 32 * 2, "flops": n * 6}
    T, K, N = case["T"], case["K"], case["N"]
    b = N * K * 17 // 32 + T * N * 2 + (T * K * 2 if case["x"] == "bf16" else T * K * 17 // 32)
    b += (N * 4 if case["bias"] else 0) + (T * N * 2 if case["residual"] else 0)
    return {"bytes": b, "flops": 2 * T * N * K}


# ---- inputs ----------------------------------------------------------------------------------

def _random_codes(g, rows, K):
    """MXFP4 rows as a calibrated weight matrix has them: every code, scales about 2^-7."""
    codes = torch.randint(0, 256, (rows, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    scales = torch.randint(118, 122, (rows, K // 32), generator=g, device=DEV, dtype=torch.uint8)
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    st = {"case": dict(case)}
    if case["op"] == "select":
        T, E, k = case["T"], case["E"], case["k"]
        st["logits"] = torch.randn(T, E, generator=g, device=DEV) * 1.7
        st["bias"] = torch.randn(E, generator=g, device=DEV) * 0.05 if case["bias"] else None
        if own:
            import routed_expert_ffn_moe_gb300 as moe

            st["shape"] = moe.shape_of(T, 7168, E, k, 2048)
            st["gate"] = moe.gate_of(case["score"], case["groups"], case["keep"], case["group_top"],
                                     case["renorm"], case["scale"])
            st["idx"] = torch.empty(T, k, dtype=torch.int32, device=DEV)
            st["w"] = torch.empty(T, k, dtype=torch.float32, device=DEV)
        return st
    if case["op"] == "quant":
        rows, K = case["rows"], case["K"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        x = torch.randn(rows, K + case["pad"], generator=g, device=DEV, dtype=dt)
        # channels of other sizes, as activations and weights have them
        x *= torch.exp2(torch.randint(-3, 4, (K + case["pad"],), generator=g, device=DEV)).to(dt)
        st["x"] = x[:, :K]
        st["back"] = torch.empty(rows, K, device=DEV, dtype=dt)
        if own:
            import routed_expert_ffn_moe_gb300 as moe

            st["rows"] = moe.mx_rows(rows, K, case["dtype"], case["tiles"], stride=K + case["pad"])
            st["back_rows"] = moe.mx_rows(rows, K, case["dtype"], case["tiles"])
            st["codes"] = torch.empty(rows, K // 2, device=DEV, dtype=torch.uint8)
            st["scales"] = torch.empty(moe.moe_mx_scale_bytes(st["rows"]), device=DEV, dtype=torch.uint8)
        return st
    T, K, N = case["T"], case["K"], case["N"]
    st["w"], st["w_scales"] = _random_codes(g, N, K)
    st["x_scales"] = None
    if case["x"] == "bf16":
        st["x"] = torch.randn(T, K, generator=g, device=DEV, dtype=torch.bfloat16)
    else:
        st["x"], st["x_scales"] = _random_codes(g, T, K)
    st["bias"] = torch.randn(N, generator=g, device=DEV) if case["bias"] else None
    st["residual"] = None
    if case["residual"]:
        st["residual"] = torch.randn(T, N, generator=g, device=DEV, dtype=torch.bfloat16)
    st["y"] = torch.empty(T, N, device=DEV, dtype=torch.bfloat16)
    if own:
        import routed_expert_ffn_moe_gb300 as moe

        def tiled(scales, rows):
            of = moe.mx_rows(rows, K, tiles=True)
            t = torch.empty(moe.moe_mx_scale_bytes(of), device=DEV, dtype=torch.uint8)
            moe.moe_mx_tile_scales(of, scales, t)
            return t

        st["w_tiles"] = tiled(st["w_scales"], N)
        st["x_tiles"] = tiled(st["x_scales"], T) if st["x_scales"] is not None else None
        st["shape"] = moe.mx_shape(T, N, K, case["x"])
        st["ws"] = torch.zeros(max(256, moe.moe_mx_linear_workspace_size(st["shape"])), device=DEV,
                               dtype=torch.uint8)
    return st


# ---- one pass --------------------------------------------------------------------------------

def run(st):
    op = st["case"]["op"]
    if own:
        return _run_own(st, op)
    return {"select": _plain_select, "quant": _plain_quant, "linear": _plain_linear}[op](st)


def _run_own(st, op):
    import routed_expert_ffn_moe_gb300 as moe

    if op == "select":
        moe.moe_route_select(st["shape"], st["gate"], st["logits"], st["bias"], st["idx"], st["w"])
        return {"idx": st["idx"], "w": st["w"]}
    if op == "quant":
        moe.moe_mx_quantize(st["rows"], st["x"], st["codes"], st["scales"])
        moe.moe_mx_dequantize(st["back_rows"], st["codes"], st["scales"], st["back"])
        return {"back": st["back"]}
    moe.moe_mx_linear(st["shape"], st["x"], st["x_tiles"], st["w"], st["w_tiles"], st["bias"],
                      st["residual"], st["y"], st["ws"])
    return {"y": st["y"]}


def _plain_select(st):
    c, l = st["case"], st["logits"].double()  # choices next to a border: 64 bits
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    if c["score"] == "sigmoid":
        s = 1 / (1 + torch.exp(-l))
    else:
        e = torch.exp(l - l.amax(1, keepdim=True))
        s = e / e.sum(1, keepdim=True)
    v = s if st["bias"] is None else s + st["bias"].double()
    if G > 1:
        by = torch.sort(v.view(T, G, E // G), dim=-1, descending=True).values
        value = by[..., :c["group_top"]].sum(-1)
        order = torch.sort(value, dim=-1, descending=True, stable=True).indices
        kept = torch.zeros(T, G, dtype=torch.bool, device=DEV)
        kept.scatter_(1, order[:, :c["keep"]], True)
        v = torch.where(kept[..., None].expand(T, G, E // G).reshape(T, E), v, -math.inf)
    idx = torch.sort(v, dim=-1, descending=True, stable=True).indices[:, :k]
    w = s.gather(1, idx)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return {"idx": idx.to(torch.int32), "w": (w * c["scale"]).float()}


def _plain_codes(x):
    """Magnitude, sign and scale exponent of rows of 32-element blocks, in 32 bits."""
    x = x.float().unflatten(-1, (-1, 32))
    amax = x.abs().amax(-1, keepdim=True)
    e = (torch.frexp(amax).exponent - 3).clamp(-127, 127)  # frexp's mantissa lies in [1/2, 1)
    e = torch.where(amax > 0, e, 0)
    a = torch.ldexp(x.abs(), -e)
    # the middle between two values goes to the one with an even code
    n = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int()
         + (a > 2.5).int() + (a >= 3.5).int() + (a > 5).int())
    return n, x < 0, e


def _plain_values(n, negative, e):
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=DEV)
    v = table[n]
    return torch.ldexp(torch.where(negative, -v, v), e).flatten(-2)


def _plain_quant(st):
    st["back"].copy_(_plain_values(*_plain_codes(st["x"])))
    return {"back": st["back"]}


def _plain_matrix(codes, scales):
    """The values of MXFP4 rows."""
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long().unflatten(-1, (-1, 32))
    return _plain_values(n & 7, n > 7, scales.int()[..., None] - 127)


def _plain_linear(st):
    x = _plain_values(*_plain_codes(st["x"])) if st["x_scales"] is None else _plain_matrix(st["x"], st["x_scales"])
    y = x @ _plain_matrix(st["w"], st["w_scales"]).t()
    if st["bias"] is not None:
        y = y + st["bias"]
    if st["residual"] is not None:
        y = y + st["residual"].float()
    st["y"].copy_(y)
    return {"y": st["y"]}


# ---- the definition in 64 bits ---------------------------------------------------------------

def _power_below(x):
    """The largest power of two that is not above x, exactly: 2 m is the mantissa in [1, 2)."""
    return x / (2 * torch.frexp(x).mantissa)


def _exact_blocks(x):
    """Nearest MXFP4 values of a matrix: a step of half a unit below 2, one below 4, two above."""
    b = x.double().reshape(x.shape[0], -1, 32)
    top = b.abs().max(-1, keepdim=True).values
    unit = _power_below(torch.where(top > 0, top, 4.0)).clamp(min=2.0 ** -125) / 4
    a = b / unit
    step = _power_below(a.abs().clamp(min=1.0)) / 2
    a = (torch.round(a / step) * step).clamp(-6, 6)
    return (a * unit).reshape(x.shape)


def _exact_codes(codes, scales):
    v = torch.empty(codes.shape[0], codes.shape[1] * 2, device=DEV, dtype=torch.float64)
    for at, c in ((0, codes % 16), (1, codes // 16)):
        ex, man = (c // 2) % 4, (c % 2).double()  # sign, two exponent bits, one mantissa bit
        mag = torch.where(ex == 0, man / 2, (1 + man / 2) * torch.exp2(ex.double() - 1))
        v[:, at::2] = torch.where(c >= 8, -mag, mag)
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, 1)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "quant":
        return {"back": _exact_blocks(st["x"])}
    if case["op"] == "linear":
        x = _exact_blocks(st["x"]) if case["x"] == "bf16" else _exact_codes(st["x"], st["x_scales"])
        y = torch.empty(case["T"], case["N"], device=DEV, dtype=torch.float64)
        for n0 in range(0, case["N"], 4096):
            n1 = min(case["N"], n0 + 4096)
            y[:, n0:n1] = torch.mm(x, _exact_codes(st["w"][n0:n1], st["w_scales"][n0:n1]).T)
        if case["bias"]:
            y += st["bias"].double()
        if case["residual"]:
            y += st["residual"].double()
        return {"y": y}
    T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
    l = st["logits"].double()
    s = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, 1)
    left = s.clone() if st["bias"] is None else s + st["bias"].double()
    by = left.view(T, G, -1).clone()
    value = torch.zeros(T, G, device=DEV, dtype=torch.float64)
    for _ in range(case["group_top"]):
        top = by.max(-1, keepdim=True)
        value += top.values[..., 0]
        by.scatter_(-1, top.indices, -math.inf)
    open_ = torch.zeros(T, G, dtype=torch.bool, device=DEV)
    rows = torch.arange(T, device=DEV)
    for _ in range(case["keep"]):  # one group, then one expert, at a time: the largest, the first of equals
        at = (value == value.max(1, keepdim=True).values).int().argmax(1)
        open_[rows, at] = True
        value[rows, at] = -math.inf
    left = left.masked_fill(~open_.repeat_interleave(E // G, 1), -math.inf)
    w = torch.empty(T, k, device=DEV, dtype=torch.float64)
    idx = torch.empty(T, k, device=DEV, dtype=torch.int32)
    for j in range(k):
        at = (left == left.max(1, keepdim=True).values).int().argmax(1)
        idx[:, j], w[:, j] = at, s[rows, at]
        left[rows, at] = -math.inf
    if case["renorm"]:
        w /= w.sum(1, keepdim=True)
    return {"idx": idx, "w": w * case["scale"]}
