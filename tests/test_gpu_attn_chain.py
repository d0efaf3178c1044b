"""Steps of the attention layer launched one behind the other, without a wait in between, give what
they give one at a time."""
import pytest
import torch

import routed_expert_ffn_moe_gb300 as moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from routed_expert_ffn_moe_gb300 import build
    build.build()
    moe.load()


@pytest.mark.parametrize("B", [1, 3, 16])
@pytest.mark.parametrize("kv,D", [("bf16", 128), ("fp8", 64)])
def test_short_decode_steps_in_a_row(B, kv, D):
    """Sequences of one tile: no item spans blocks, so k_attn_join has nothing to do, while the step
    behind it overwrites the queries, the cache and the output."""
    Hq, Hkv, steps = 8, 2, 60
    torch.manual_seed(3)
    qkv = torch.randn(steps, B, (Hq + 2 * Hkv) * D, device="cuda").to(torch.bfloat16)
    table = torch.randperm(4 * B, device="cuda").to(torch.int32).view(B, 4)
    lens = [(torch.arange(B, device="cuda") % 4 + n + 1).clamp(max=60).to(torch.int32)
            for n in range(steps)]

    def run(wait):
        layer = moe.AttnLayer(Hq, Hkv, D, num_pages=4 * B, max_pages=4, max_batch=B, max_tokens=B,
                              kv_dtype=kv)
        out = torch.empty(steps, B, Hq * D, dtype=torch.bfloat16, device="cuda")
        for n in range(steps):
            out[n].copy_(layer.forward(qkv[n], table, lens[n]))
            # once more, with the next step right behind it: no copy in between
            layer.forward(qkv[n], table, lens[n])
            if wait:
                torch.cuda.synchronize()
        layer.check()
        return out, layer.k_cache, layer.v_cache

    one, row = run(True), run(False)
    for a, b in zip(one, row):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("D", [64, 128])
def test_prefill_calls_in_a_row(D):
    """Blocks of one call make room for the next one's while their last products end: the same bits as
    one call at a time."""
    from attn_helpers import Step, workspace

    steps = [Step(lens=[n], new=[m], Hq=8, Hkv=2, D=D, page=64, seed=n)
             for n, m in ((1, 1), (70, 70), (300, 5), (5000, 3), (900, 700))]
    calls = []
    for s in steps:
        t, shape = s.device(), s.shape()
        o = torch.empty(s.T, 8, D, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(s.T, 8, device="cuda")
        ws = workspace(shape, True)
        calls.append((o, lse, ws, lambda t=t, sh=shape, o=o, lse=lse, ws=ws: moe.moe_attn_prefill(
            sh, t["q"], t["k"], t["v"], None, None, t["table"], t["lens"], t["q_start"], o, lse, ws)))
    one = []
    for o, lse, _, call in calls:
        call()
        torch.cuda.synchronize()
        one.append((o.clone(), lse.clone()))
        o.fill_(float("nan"))
    for _ in range(100):
        for c in calls:
            c[3]()
    torch.cuda.synchronize()
    for (o, lse, ws, _), (o1, lse1) in zip(calls, one):
        moe.moe_check_device_status(ws)
        assert torch.equal(o.view(torch.int16), o1.view(torch.int16))
        assert torch.equal(lse, lse1)
