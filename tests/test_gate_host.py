"""Host-side checks of scored routing: every bad argument is refused before a launch (no GPU)."""
import ctypes

import pytest

import routed_expert_ffn_moe_gb300 as moe
from routed_expert_ffn_moe_gb300 import build as moe_build

F = 0x7F0000000000  # never dereferenced: every call below fails host validation


@pytest.fixture(scope="module", autouse=True)
def _lib():
    moe_build.build()
    moe.load()


def shape(**kw):
    base = dict(T=4, d=256, E=64, k=8, f=128)
    base.update(kw)
    return moe.shape_of(**base)


BAD = [
    ({}, dict(score=2), "score=2"), ({}, dict(score=-1), "score=-1"),
    ({}, dict(n_group=0), "n_group=0"), ({}, dict(n_group=33), "n_group=33"),
    ({}, dict(n_group=64), "n_group=64"), ({}, dict(n_group=5), "n_group=5"),
    ({}, dict(n_group=8, topk_group=0), "topk_group=0"),
    ({}, dict(n_group=8, topk_group=9), "topk_group=9"),
    ({}, dict(n_group=16, topk_group=1), "k=8"), ({}, dict(group_top=0), "group_top=0"),
    ({}, dict(group_top=3), "group_top=3"),
    (dict(E=32, k=4), dict(n_group=32, topk_group=4), "group_top=2"),
    ({}, dict(scale=float("nan")), "scale"), ({}, dict(scale=float("inf")), "scale"),
    (dict(k=33), {}, "k=33"), (dict(E=0), {}, "E=0"), (dict(T=-1), {}, "T=-1"),
]


@pytest.mark.parametrize("skw,gkw,word", BAD, ids=[str((b[0], b[1])) for b in BAD])
def test_bad_gates_are_refused(skw, gkw, word):
    s, g = shape(**skw), moe.gate_of(**gkw)
    with pytest.raises(moe.MoeError) as ei:
        moe.moe_route_select(s, g, F, F, F, F, stream=0)
    assert ei.value.status == -1 and word in str(ei.value)
    with pytest.raises(moe.MoeError) as ei:
        moe.moe_route_gate(s, g, F, F, F, F, F, F, F, stream=0, ws_bytes=1 << 40)
    assert ei.value.status == -1 and word in str(ei.value)


@pytest.mark.parametrize("at,word", [(0, "logits"), (2, "topk_idx"), (3, "topk_w")])
def test_null_and_misaligned_pointers(at, word):
    for bad, says in ((None, "NULL"), (F + 4, "aligned")):
        args = [F, F, F, F]
        args[at] = bad
        with pytest.raises(moe.MoeError) as ei:
            moe.moe_route_select(shape(), moe.gate_of(), *args, stream=0)
        assert word in str(ei.value) and says in str(ei.value)
    with pytest.raises(moe.MoeError, match="sel_bias"):
        moe.moe_route_select(shape(), moe.gate_of(), F, F + 4, F, F, stream=0)


def test_gate_needs_its_workspace():
    s = shape()
    n = moe.moe_workspace_size(s)
    with pytest.raises(moe.MoeError) as ei:
        moe.moe_route_gate(s, moe.gate_of(), F, F, None, None, F, F, F, stream=0, ws_bytes=n - 1)
    assert ei.value.status == -3
    for i, word in ((0, "x"), (1, "wg"), (4, "topk_idx"), (5, "topk_w"), (6, "ws")):
        args = [F, F, None, None, F, F, F]
        args[i] = None
        with pytest.raises(moe.MoeError, match=word + " is NULL"):
            moe.moe_route_gate(s, moe.gate_of(), *args, stream=0, ws_bytes=n)
    rc = moe.load().moe_route_select(ctypes.byref(s), None, F, None, F, F, None)
    assert rc == -1 and "gate is NULL" in moe.moe_last_error_string()


def test_no_tokens_is_no_call():
    moe.moe_route_select(shape(T=0), moe.gate_of(), None, None, None, None, stream=0)
