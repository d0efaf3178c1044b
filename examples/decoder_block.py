"""A decoder block on one GPU: attention over a paged cache, then the MoE FFN.

    python examples/decoder_block.py

Two sequences get their prompts in one ragged step, then tokens one at a time. Every step runs
    h = x + W_o attention(W_qkv norm(x));   y = h + moe(norm(h))
with AttnLayer (norms, rotation, append, attention) and MoeLayer; the projections are torch
matrix products, or MxLinear with `fp4`, when the experts are MXFP4 as well and the router is one of
sigmoid scores, groups and a selection bias. At the end the same tokens go through the block once more, as one prompt a
sequence, and the outputs are compared.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import routed_expert_ffn_moe_gb300 as moe  # noqa: E402


class PagePool:
    """Pages of the cache and the table of those that each sequence holds."""

    def __init__(self, num_pages, page_size, max_pages, batch):
        self.free = list(range(num_pages))[::-1]
        self.page_size, self.max_pages = page_size, max_pages
        self.pages = [[] for _ in range(batch)]
        self.lens = [0] * batch

    def grow(self, new):
        """`new` more tokens for each sequence: the table and the lengths of the step."""
        for b, n in enumerate(new):
            self.lens[b] += n
            while len(self.pages[b]) * self.page_size < self.lens[b]:
                self.pages[b].append(self.free.pop())
        table = torch.full((len(new), self.max_pages), -1, dtype=torch.int32)
        for b, pages in enumerate(self.pages):
            table[b, :len(pages)] = torch.tensor(pages, dtype=torch.int32)
        return table.cuda(), torch.tensor(self.lens, dtype=torch.int32).cuda()


class DecoderBlock:
    def __init__(self, d=512, Hq=8, Hkv=2, D=64, E=8, k=2, f=256, kv_dtype="bf16", window=0,
                 n_sink=0, fp4=False, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def w(*shape, scale=0.03):
            return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)

        self.d, self.E, self.k, self.f = d, E, k, f
        self.attn_kw = dict(Hq=Hq, Hkv=Hkv, D=D, kv_dtype=kv_dtype, window=window, n_sink=n_sink,
                            norms=(1 + w(D), 1 + w(D)))
        if kv_dtype == "fp8":  # unit-variance keys and values: about 8 deviations to the last code
            s = torch.full((Hkv,), 8 / 448, device="cuda")
            self.attn_kw["scales"] = (s, s.clone())
        self.w_qkv, self.w_o = w((Hq + 2 * Hkv) * D, d), w(d, Hq * D)
        self.moe_w = {"wg": w(E, d), "bias": None, "w13": w(E + 1, 2 * f, d), "w2": w(E + 1, d, f),
                      "s13": None, "s2": None}
        self.moe_layers, self.fp4 = {}, fp4
        if fp4:
            self.qkv = moe.MxLinear.from_weight(self.w_qkv, max_tokens=512)
            self.out = moe.MxLinear.from_weight(self.w_o, max_tokens=512)
            self.moe_w["sel_bias"] = torch.randn(E, generator=g, device="cuda") * 0.02
            for i, rows, K in (("13", 2 * f, d), ("2", d, f)):
                codes = torch.empty(E + 1, rows, K // 2, dtype=torch.uint8, device="cuda")
                scales = torch.empty(E + 1, rows, K // 32, dtype=torch.uint8, device="cuda")
                moe.moe_mx_quantize(moe.mx_rows((E + 1) * rows, K), self.moe_w["w" + i], codes, scales)
                self.moe_w["w" + i], self.moe_w["s" + i] = codes, scales

    def attention(self, **kw):
        return moe.AttnLayer(**self.attn_kw, **kw)

    def _moe(self, x):
        T = x.shape[0]
        if T not in self.moe_layers:
            gate = moe.gate_of(n_group=4, topk_group=2, scale=2.5) if self.fp4 else None
            self.moe_layers[T] = moe.MoeLayer(T, self.d, self.E, self.k, self.f, 1,
                                              "mxfp4" if self.fp4 else "bf16", self.moe_w, gate=gate)
        return self.moe_layers[T].forward(x)

    @staticmethod
    def _norm(x):
        x = x.float()
        return (x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)

    def step(self, attn, x, table, kv_len, q_start=None):
        """One step of the block: x [T, d] bf16 -> [T, d] bf16."""
        if self.fp4:
            qkv = self.qkv.forward(self._norm(x))
            h = self.out.forward(attn.forward(qkv, table, kv_len, q_start), residual=x)
            return h + self._moe(self._norm(h))
        qkv = self._norm(x) @ self.w_qkv.T
        h = x + attn.forward(qkv, table, kv_len, q_start) @ self.w_o.T
        return h + self._moe(self._norm(h))


def run(prompts=(37, 90), steps=6, page_size=16, **kw):
    """Prompts and single tokens against whole prompts: the largest relative difference of a row."""
    block = DecoderBlock(**kw)
    B, total = len(prompts), [n + steps for n in prompts]
    max_pages = -(-max(total) // page_size)
    tokens = [torch.randn(n, block.d, device="cuda").to(torch.bfloat16) for n in total]

    def layer():
        pool = PagePool(2 * B * max_pages, page_size, max_pages, B)
        return pool, block.attention(num_pages=2 * B * max_pages, page_size=page_size,
                                     max_pages=max_pages, max_batch=B, max_tokens=sum(total))

    def prompt(pool, attn, new):
        table, lens = pool.grow(new)
        q_start = torch.tensor([0] + list(new)).cumsum(0).to(torch.int32).cuda()
        x = torch.cat([t[:n] for t, n in zip(tokens, new)])
        return list(block.step(attn, x, table, lens, q_start).split(list(new)))

    pool, attn = layer()
    out = [[y] for y in prompt(pool, attn, prompts)]
    for i in range(steps):
        table, lens = pool.grow([1] * B)
        x = torch.stack([tokens[b][prompts[b] + i] for b in range(B)])
        for b, y in enumerate(block.step(attn, x, table, lens)):
            out[b].append(y[None])
    attn.check()
    pool, attn = layer()
    whole = prompt(pool, attn, total)
    attn.check()
    worst = 0.0
    for b in range(B):
        a, c = torch.cat(out[b]).float(), whole[b].float()
        worst = max(worst, ((a - c).norm(dim=-1) / c.norm(dim=-1)).max().item())
    return worst


if __name__ == "__main__":
    torch.manual_seed(0)
    for kw in ({}, {"kv_dtype": "fp8"}, {"window": 48, "n_sink": 4}, {"fp4": True}):
        print(kw or "bf16 cache", "steps against whole prompts: largest relative difference",
              f"{run(**kw):.2e}")
