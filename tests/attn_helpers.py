"""The attention operators in 64 bits (torch, CPU), their error bounds, and the inputs of their
tests: paged caches in any stride order whose unused places hold NaN."""
from __future__ import annotations

import math
from dataclasses import dataclass, field

import torch

import routed_expert_ffn_moe_gb300 as moe

F64 = torch.float64


def half_ulp(x, bits, min_exp):
    """Half the spacing at |x| of a format with `bits` significant bits and smallest normal
    2^min_exp."""
    a = x.abs().clamp(min=2.0 ** min_exp)
    return 2.0 ** (torch.floor(torch.log2(a)) - bits)


def half_ulp_bf16(x):
    return half_ulp(x, 8, -126)


def half_ulp_e4m3(x):
    return half_ulp(x, 4, -6)


@dataclass
class Step:
    """One step of a batch: its shape and everything the operators take, on the GPU."""
    lens: list
    new: list
    Hq: int
    Hkv: int
    D: int = 128
    kv: str = "bf16"
    page: int = 16
    order: str = "HND"        # or "NHD", or "gaps": padded strides
    window: int = 0
    sink: int = 0
    seed: int = 0
    scales: bool = True
    spread: float = 1.0       # standard deviation of the queries
    extra_pages: int = 2
    t: dict = field(default_factory=dict)

    def __post_init__(self):
        g = torch.Generator().manual_seed(self.seed)
        B, T = len(self.lens), sum(self.new)
        D, Hkv, page = self.D, self.Hkv, self.page
        need = [-(-n // page) for n in self.lens]
        self.num_pages = sum(need) + self.extra_pages
        self.max_pages = max(max(need, default=0), 1)
        table = torch.full((B, self.max_pages), -1, dtype=torch.int32)
        perm = torch.randperm(self.num_pages, generator=g).to(torch.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = perm[at:at + n]
            at += n
        self.table = table
        if self.order == "HND":
            size, self.strides = (self.num_pages, Hkv, page, D), (0, 0, 0)
            view = lambda x: x                                              # noqa: E731
        elif self.order == "NHD":
            size = (self.num_pages, page, Hkv, D)
            self.strides = (page * Hkv * D, D, Hkv * D)
            view = lambda x: x.permute(0, 2, 1, 3)                          # noqa: E731
        else:  # gaps between tokens, heads and pages
            size = (self.num_pages + 1, Hkv + 1, page + 1, D + 16)
            self.strides = ((Hkv + 1) * (page + 1) * (D + 16), (page + 1) * (D + 16), D + 16)
            view = lambda x: x[:self.num_pages, :Hkv, :page, :D]            # noqa: E731
        self.k_scale = self.v_scale = None
        if self.kv == "fp8" and self.scales:
            self.k_scale = torch.rand(Hkv, generator=g) * 0.02 + 0.01
            self.v_scale = torch.rand(Hkv, generator=g) * 0.02 + 0.01
        dt = torch.bfloat16 if self.kv == "bf16" else torch.float8_e4m3fn
        self.caches = []
        for sc in (self.k_scale, self.v_scale):
            raw = torch.full(size, float("nan"), dtype=torch.float32)
            v = view(raw)
            for b, n in enumerate(self.lens):
                x = torch.randn(n, Hkv, D, generator=g)
                if sc is not None:
                    x = x / sc[:, None]
                for i in range(need[b]):
                    m = min(page, n - i * page)
                    v[int(table[b, i]), :, :m] = x[i * page:i * page + m].transpose(0, 1)
            self.caches.append(raw.to(dt))
        self.k_view, self.v_view = (view(c) for c in self.caches)
        self.q_start = torch.tensor([0] + self.new).cumsum(0).to(torch.int32)
        self.q = (torch.randn(T, self.Hq, D, generator=g) * self.spread).to(torch.bfloat16)
        self.B, self.T = B, T

    def shape(self, **more):
        kw = dict(page_stride=self.strides[0], head_stride=self.strides[1],
                  token_stride=self.strides[2], window=self.window, n_sink=self.sink)
        kw.update(more)
        return moe.attn_shape(T=self.T, B=self.B, Hq=self.Hq, Hkv=self.Hkv, D=self.D,
                              kv_dtype=self.kv, page_size=self.page, max_pages=self.max_pages,
                              num_pages=self.num_pages, **kw)

    def device(self):
        """The tensors on the GPU (made once)."""
        if not self.t:
            up = lambda x: None if x is None else x.cuda()                  # noqa: E731
            self.t = dict(q=up(self.q), k=up(self.caches[0]), v=up(self.caches[1]),
                          ks=up(self.k_scale), vs=up(self.v_scale), table=up(self.table),
                          lens=torch.tensor(self.lens, dtype=torch.int32).cuda(),
                          q_start=up(self.q_start))
        return self.t

    # ---- the definition ----

    def cached(self, b):
        """k and v of sequence b in 64 bits, scales applied: [n, Hkv, D] each."""
        n, out = self.lens[b], []
        for view, sc in ((self.k_view, self.k_scale), (self.v_view, self.v_scale)):
            j = torch.arange(n)
            x = view.float()[self.table[b, j // self.page].long(), :, j % self.page].to(F64)
            out.append(x if sc is None else x * sc.to(F64)[:, None])
        return out

    def reference(self, p_round=2.0 ** -9):
        """o, lse in 64 bits and their bounds: see attention_bounds."""
        o = torch.zeros(self.T, self.Hq, self.D, dtype=F64)
        lse = torch.full((self.T, self.Hq), -math.inf, dtype=F64)
        o_tol, lse_tol = torch.zeros_like(o), torch.zeros_like(lse)
        G, scale, t0 = self.Hq // self.Hkv, 1 / math.sqrt(self.D), 0
        for b, (n, new) in enumerate(zip(self.lens, self.new)):
            if new and n:
                k, v = self.cached(b)
                q = self.q[t0:t0 + new].to(F64).view(new, self.Hkv, G, self.D)
                s = torch.einsum("thgd,jhd->thgj", q, k) * scale
                big = torch.einsum("thgd,jhd->thgj", q.abs(), k.abs()).amax(-1) * scale
                pos = (n - new + torch.arange(new))[:, None]
                j = torch.arange(n)[None, :]
                seen = j <= pos
                if self.window:
                    seen &= (pos - j < self.window) | (j < self.sink)
                s = s.masked_fill(~seen[:, None, None, :], -math.inf)
                some = seen.any(-1)
                L = torch.logsumexp(s, -1)
                p = torch.exp(s - L[..., None]).nan_to_num(0.0)
                y = torch.einsum("thgj,jhd->thgd", p, v)
                yabs = torch.einsum("thgj,jhd->thgd", p, v.abs())
                e_o, e_l = attention_bounds(y, yabs, big, n, L, p_round)
                for dst, src in ((o, y), (o_tol, e_o)):
                    dst[t0:t0 + new] = torch.where(some[:, None, None], src.reshape(new, self.Hq, self.D), 0.0)
                lse[t0:t0 + new] = L.reshape(new, self.Hq)
                lse_tol[t0:t0 + new] = e_l.reshape(new, self.Hq)
            t0 += new
        return o, lse, o_tol, lse_tol


def attention_bounds(y, yabs, big, n, lse, p_round=2.0 ** -9):
    """Bounds of |o - y| and |lse error| for an output y = sum p v.

    A score is a sum of D <= 128 exact products in fp32: within 128 * 2^-24 of the sum of their
    magnitudes (`big`: the largest over the keys, scale included), and its scaling adds 2^-22 of it.
    Each e^s carries that and 2^-21 of its own (base-2 exponential and its argument); a
    probability enters the product within `p_round` of itself (l is summed before that rounding),
    so numerator and l together move y by at most (p_round + 2 e) sum p |v|. fp32 sums over n keys
    (at most n/8 + 64 in a row) add their own, and the result is rounded to bf16."""
    e = big * (2.0 ** -17 + 2.0 ** -22) + 2.0 ** -21
    sums = (n / 8 + 64) * 2.0 ** -24
    o_tol = half_ulp_bf16(y) * 1.01 + (p_round + 2 * e + 2 * sums)[..., None] * yabs + 1e-30
    lse_tol = e + sums + lse.abs() * 2.0 ** -22
    return o_tol, lse_tol.nan_to_num(0.0)


def workspace(shape, prefill=False):
    ws = torch.empty(moe.moe_attn_workspace_size(shape, prefill), dtype=torch.uint8, device="cuda")
    ws.fill_(0xA5)
    ws[:moe.moe_attn_workspace_zero_bytes()].zero_()
    return ws


def check_attention(step, o, lse, what="", p_round=2.0 ** -9):
    ref, ref_lse, o_tol, lse_tol = step.reference(p_round)
    o, lse = o.cpu().to(F64), lse.cpu().to(F64)
    assert torch.isfinite(o).all(), (what, "o is not finite")
    over = (o - ref).abs() - o_tol
    assert over.max().item() <= 0, (what, over.max().item(), (o - ref).abs().max().item())
    none = torch.isinf(ref_lse)
    assert torch.equal(torch.isinf(lse) & (lse < 0), none), (what, "rows that see nothing")
    over = ((lse - ref_lse).abs() - lse_tol)[~none]
    assert over.numel() == 0 or over.max().item() <= 0, (what, over.max().item())


# ---- append ----------------------------------------------------------------------------------

def rotate64(x, cos, sin, pairs):
    """x [..., D] in 64 bits, cos and sin [..., rot/2] broadcast over heads."""
    half = cos.shape[-1]
    y = x.clone()
    lo, hi = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if pairs else (
        slice(0, half), slice(half, 2 * half))
    a, b = x[..., lo], x[..., hi]
    y[..., lo], y[..., hi] = a * cos - b * sin, b * cos + a * sin
    return y


def norm64(x, w, eps):
    if w is None:
        return x
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.to(F64)
