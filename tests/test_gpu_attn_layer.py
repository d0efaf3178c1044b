"""AttnLayer and the decoder block example: prompts and single tokens give what whole prompts give."""
import importlib.util
import os

import pytest
import torch

import routed_expert_ffn_moe_gb300 as moe

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from routed_expert_ffn_moe_gb300 import build
    build.build()
    moe.load()


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location(
        "decoder_block", os.path.join(ROOT, "examples", "decoder_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


# Both ways round the same values to bf16 at the same places, but sum in other orders: a rounding
# that falls the other way moves a row by up to 2^-8 of an element, a few times over along the
# block (qkv, attention, two residual sums, MoE), and the experts' choice by nothing unless two
# logits are that close: the seeds here have none.
BOUND = 4 * 2.0 ** -8


@pytest.mark.parametrize("kw", [
    dict(), dict(kv_dtype="fp8"), dict(window=48, n_sink=4), dict(D=128, Hq=4, Hkv=1),
    dict(prompts=(1, 200, 17), steps=3, page_size=7, Hq=14, d=896, D=64),
], ids=str)
def test_steps_agree_with_whole_prompts(example, kw):
    torch.manual_seed(1)
    assert example.run(**kw) <= BOUND


def test_layer_refuses_what_it_was_not_made_for():
    layer = moe.AttnLayer(4, 2, 64, num_pages=8, max_pages=4, max_batch=2, max_tokens=16)
    table = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    lens = torch.ones(2, dtype=torch.int32, device="cuda")
    qkv = torch.zeros(17, 8 * 64, dtype=torch.bfloat16, device="cuda")
    start = torch.tensor([0, 16, 17], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="17 tokens"):
        layer.forward(qkv, table, lens, start)
    with pytest.raises(ValueError, match="3 sequences"):
        layer.forward(qkv[:3], table[:1].expand(3, 4), lens[:1].expand(3))
    with pytest.raises(ValueError, match="tables of 3 pages"):
        layer.forward(qkv[:2], table[:, :3], lens)
    with pytest.raises(moe.MoeError) as ei:
        moe.AttnLayer(4, 2, 96, num_pages=8)
    assert "D=96" in str(ei.value)


def test_layer_in_a_cuda_graph():
    # a decode step captured once and replayed as the lengths grow
    layer = moe.AttnLayer(8, 2, 128, num_pages=40, max_pages=20, max_batch=2, max_tokens=64)
    torch.manual_seed(2)
    qkv = torch.randn(2, 12 * 128, device="cuda").to(torch.bfloat16)
    table = torch.arange(40, dtype=torch.int32, device="cuda").view(2, 20)
    lens = torch.tensor([1, 5], dtype=torch.int32, device="cuda")
    layer.forward(qkv, table, lens)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = layer.forward(qkv, table, lens)
    for n in range(1, 40):
        lens.copy_(torch.tensor([n, n + 4], dtype=torch.int32))
        qkv.copy_(torch.randn(2, 12 * 128, device="cuda").to(torch.bfloat16))
        graph.replay()
        got = o.clone()
        again = layer.forward(qkv, table, lens)
        assert torch.equal(got.view(torch.int16), again.view(torch.int16)), n
    layer.check()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_layer_takes_rows_that_lie_apart(kv):
    # a projection that has more columns than the layer needs, and arrays made for larger batches
    torch.manual_seed(4)
    row, T = 12 * 128, 50
    wide = torch.randn(T, row + 64, device="cuda").to(torch.bfloat16)
    table = torch.arange(12, dtype=torch.int32, device="cuda").view(3, 4)
    lens = torch.tensor([40, 11], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 40, 50, 99, 99], dtype=torch.int32, device="cuda")
    out = []
    for qkv in (wide[:, :row], wide[:, :row].contiguous(), wide[:, :row].reshape(T, 12, 128)):
        layer = moe.AttnLayer(8, 2, 128, num_pages=12, max_pages=4, max_batch=4, max_tokens=64,
                              kv_dtype=kv)
        lse = torch.zeros(T, 8, device="cuda")
        o = layer.forward(qkv, table, lens, start, lse=lse)
        one = layer.forward(qkv[:2], table, lens + 1)
        layer.check()
        out.append((o.clone(), one.clone(), lse, layer.k_cache, layer.v_cache))
    for other in out[1:]:
        for a, b in zip(out[0], other):
            assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
