"""What AttnLayer.forward refuses before it hands pointers to the library: tensors of another type or
layout would be read, and pages written, at wrong places without a word. The layer and its tensors lie
in host memory here; every call is refused before a launch."""
import pytest
import torch

import routed_expert_ffn_moe_gb300 as moe
from routed_expert_ffn_moe_gb300 import build as moe_build

HQ, HKV, D, PAGES = 4, 2, 64, 4
ROW = (HQ + 2 * HKV) * D
I32, BF16 = torch.int32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    moe_build.build()
    moe.load()


@pytest.fixture(scope="module")
def layer():
    return moe.AttnLayer(HQ, HKV, D, num_pages=8, max_pages=PAGES, max_batch=4, max_tokens=16,
                         device="cpu")


def good(**kw):
    args = dict(qkv=torch.zeros(6, ROW, dtype=BF16), block_table=torch.zeros(2, PAGES, dtype=I32),
                kv_len=torch.ones(2, dtype=I32), q_start=torch.tensor([0, 5, 6], dtype=I32))
    args.update(kw)
    return args


BAD = [
    ("qkv", torch.zeros(6, ROW)),                                       # fp32
    ("qkv", torch.zeros(6, ROW, dtype=torch.float16)),
    ("qkv", torch.zeros(6, ROW - D, dtype=BF16)),                       # too narrow
    ("qkv", torch.zeros(6, ROW + D, dtype=BF16)),                       # too wide
    ("qkv", torch.zeros(ROW, 6, dtype=BF16).t()),                       # columns apart
    ("qkv", torch.zeros(1, ROW, dtype=BF16).expand(6, ROW)),            # one row for all
    ("qkv", torch.zeros(6, 2 * ROW // D, D, dtype=BF16)[:, ::2]),       # heads apart
    ("block_table", torch.zeros(2, PAGES, dtype=torch.int64)),          # torch's default
    ("block_table", torch.zeros(2, PAGES + 3, dtype=I32)[:, :PAGES]),   # columns of a wider one
    ("block_table", torch.zeros(PAGES, 2, dtype=I32).t()),
    ("block_table", torch.zeros(1, PAGES, dtype=I32)),                  # too few rows
    ("kv_len", torch.ones(2, dtype=torch.int64)),
    ("kv_len", torch.ones(4, dtype=I32)[::2]),
    ("q_start", torch.tensor([0, 5, 6])),
    ("q_start", torch.tensor([0, 5], dtype=I32)),                       # no end
    ("q_start", torch.zeros(6, dtype=I32)[::2]),
    ("positions", torch.zeros(6, dtype=torch.int64)),
    ("positions", torch.zeros(5, dtype=I32)),
    ("lse", torch.zeros(6, HQ, dtype=torch.float64)),
    ("lse", torch.zeros(6, HQ - 1)),
    ("lse", torch.zeros(HQ, 6).t()),
]


@pytest.mark.parametrize("name,value", BAD, ids=[f"{n}-{i}" for i, (n, _) in enumerate(BAD)])
def test_wrong_tensors_are_refused(layer, name, value):
    with pytest.raises(ValueError, match=name):
        layer.forward(**good(**{name: value}))


def test_tensors_of_another_device_are_refused(layer):
    meta = torch.zeros(2, dtype=I32, device="meta")
    with pytest.raises(ValueError, match="kv_len"):
        layer.forward(**good(kv_len=meta))


@pytest.mark.parametrize("kw,word", [
    (dict(norms=(torch.ones(D), torch.ones(D))), "q_norm"),                       # fp32
    (dict(norms=(torch.ones(D, dtype=BF16), torch.ones(D // 2, dtype=BF16))), "k_norm"),
    (dict(kv_dtype="fp8", scales=(torch.ones(HKV, dtype=BF16), torch.ones(HKV))), "k_scale"),
    (dict(kv_dtype="fp8", scales=(torch.ones(HKV), torch.ones(1))), "v_scale"),
], ids=lambda v: v if isinstance(v, str) else "")
def test_wrong_weights_are_refused(kw, word):
    with pytest.raises(ValueError, match=word):
        moe.AttnLayer(HQ, HKV, D, num_pages=8, max_pages=PAGES, max_batch=4, max_tokens=16,
                      device="cpu", **kw)


@pytest.mark.parametrize("name,number,dtype", [("bf16", moe.MOE_KV_BF16, BF16),
                                               ("fp8", moe.MOE_KV_FP8_E4M3, torch.uint8)])
def test_the_cache_holds_what_its_type_needs(name, number, dtype):
    # the type by its name or by the library's number
    for kv in (name, number):
        layer = moe.AttnLayer(HQ, HKV, D, num_pages=8, max_pages=PAGES, max_batch=4, max_tokens=16,
                              kv_dtype=kv, device="cpu")
        assert layer.k_cache.dtype == dtype and layer.v_cache.dtype == dtype
