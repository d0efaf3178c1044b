"""GPU: scored routing of large batches from the tokens, whose logits are formed in their defined order only where the
choice depends on them, against the routing that forms all of them: the same experts, at every score,
grouping, bias and size, with ties, masks, infinities and NaNs. No formed logit may leave its bound."""
import numpy as np
import pytest

import routed_expert_ffn_moe_gb300 as moe
from gpu_helpers import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from routed_expert_ffn_moe_gb300 import build
    build.build()
    moe.load()


def route(monkeypatch, always, x, wg, bias, sel, k, gate):
    t = torch()
    monkeypatch.setenv("MOE_ROUTER_TC_MIN_TOKENS", "1" if always else "1000000000")
    s = moe.shape_of(x.shape[0], x.shape[1], wg.shape[0], k, 128)
    ws = t.full((moe.moe_workspace_size(s),), 255, dtype=t.uint8, device="cuda")
    idx = t.full((x.shape[0], k), -7, dtype=t.int32, device="cuda")
    w = t.full((x.shape[0], k), -7.0, device="cuda")
    moe.moe_route_gate(s, moe.gate_of(**gate), x, wg, bias, sel, idx, w, ws)
    moe.moe_check_device_status(ws)
    status = ws[:12].view(t.int32).cpu().numpy()
    return idx.cpu().numpy(), w.cpu().numpy(), status


def check(monkeypatch, x, wg, bias, sel, k, full=0, **gate):
    """`full`: the tokens all of whose logits were formed, None for any number."""
    i, w, st = route(monkeypatch, True, x, wg, bias, sel, k, gate)
    ri, rw, _ = route(monkeypatch, False, x, wg, bias, sel, k, gate)
    np.testing.assert_array_equal(i, ri)
    np.testing.assert_array_equal(np.isnan(w), np.isnan(rw))
    ok = ~np.isnan(rw)
    # of the same k logits: the sums of 32 scores may be taken in another order, 31 roundings each
    assert (np.abs(w - rw)[ok] <= 64 * 2.0 ** -24 * np.abs(rw[ok])).all()
    if full is not None:
        assert st[1] == full
        assert 0.0 <= float(np.array([st[2]], np.int32).view(np.float32)[0]) < 1.0 / 16
    return i, w


def draw(T, d, E, seed):
    t = torch()
    g = t.Generator(device="cuda").manual_seed(seed)
    x = t.randn(T, d, generator=g, device="cuda", dtype=t.bfloat16)
    wg = (t.randn(E, d, generator=g, device="cuda") * (2.0 / d ** 0.5)).to(t.bfloat16)
    bias = t.randn(E, generator=g, device="cuda") * 0.3
    sel = t.randn(E, generator=g, device="cuda") * 0.1
    return x, wg, bias, sel


GATES = [dict(score="sigmoid"), dict(score="sigmoid", renorm=False, scale=2.5),
         dict(score="sigmoid", n_group=8, topk_group=4, scale=2.5),
         dict(score="sigmoid", n_group=8, topk_group=3, group_top=1),
         dict(score="sigmoid", n_group=32, topk_group=5), dict(score="sigmoid", n_group=4, topk_group=4),
         dict(score="softmax"), dict(score="softmax", n_group=16, topk_group=3, group_top=1),
         dict(score="softmax", n_group=8, topk_group=4), dict(score="softmax", renorm=False)]


@pytest.mark.parametrize("gate", GATES, ids=str)
@pytest.mark.parametrize("with_bias,with_sel", [(False, False), (True, False), (False, True), (True, True)])
def test_same_choice_as_with_every_logit(monkeypatch, gate, with_bias, with_sel):
    x, wg, bias, sel = draw(1501, 1024, 256, 5)
    settled = gate["score"] == "sigmoid" or (
        not with_sel and gate.get("renorm", True) and ("n_group" not in gate or gate.get("group_top") == 1))
    check(monkeypatch, x, wg, bias if with_bias else None, sel if with_sel else None, 8,
          full=0 if settled else None, **gate)


@pytest.mark.parametrize("T,d,E,k,G,keep", [
    (1, 128, 128, 1, 1, 1), (3, 128, 128, 32, 4, 1), (130, 7168, 256, 8, 8, 4), (65, 16384, 128, 4, 16, 5),
    (70, 1024, 1024, 32, 32, 9), (257, 640, 640, 7, 5, 2), (500, 512, 384, 6, 3, 2), (9, 512, 896, 9, 28, 27)])
def test_sizes(monkeypatch, T, d, E, k, G, keep):
    x, wg, bias, sel = draw(T, d, E, T)
    for top in (1, 2):
        check(monkeypatch, x, wg, bias, sel, k, n_group=G, topk_group=keep, group_top=top)
        check(monkeypatch, x, wg, None, None, k, n_group=G, topk_group=keep, group_top=top)


def test_ties_and_choices_a_hair_apart(monkeypatch):
    t = torch()
    x, wg, bias, sel = draw(600, 512, 256, 8)
    wg[128:] = wg[:128]
    wg[129::2, 7] *= 1 + 2.0 ** -7  # one step in one element of every other row
    x[:4] = 0
    sel[128:] = sel[:128]
    bias[128:] = bias[:128]
    for gate in (dict(), dict(n_group=8, topk_group=4), dict(n_group=8, topk_group=4, group_top=1)):
        check(monkeypatch, x, wg, bias, sel, 8, **gate)
        check(monkeypatch, x, wg, None, None, 8, **gate)
    sel = t.zeros_like(sel)
    check(monkeypatch, x * 0.001, wg, None, sel, 8, n_group=8, topk_group=4)
    check(monkeypatch, x * 64, wg, None, sel, 8, n_group=8, topk_group=4)  # scores of 1


def test_masks_infinities_and_nans(monkeypatch):
    x, wg, bias, sel = draw(300, 512, 256, 9)
    inf, nan = float("inf"), float("nan")
    grouped = dict(n_group=8, topk_group=4)
    for gate in (dict(), grouped, dict(grouped, group_top=1), dict(score="softmax")):
        b = sel.clone()
        b[::3] = -inf
        check(monkeypatch, x, wg, bias, b, 8, full=0 if "score" not in gate else None, **gate)
        b[32:64] = nan
        b[65] = inf
        check(monkeypatch, x, wg, bias, b, 8, full=None, **gate)
        b[:] = -inf
        check(monkeypatch, x, wg, bias, b, 8, full=None, **gate)
        lb = bias.clone()
        lb[5::2] = -inf
        check(monkeypatch, x, wg, lb, None, 8, full=0, **gate)  # a masked logit needs no sum
        lb[9] = nan
        check(monkeypatch, x, wg, lb, sel, 8, full=None, **gate)
        y = x.clone()
        y[3, 5], y[4, 6], y[5, :] = inf, nan, 3e38
        check(monkeypatch, y, wg, bias, sel, 8, full=None, **gate)
        check(monkeypatch, y, wg, None, None, 8, full=None, **gate)


def test_zeros_and_values_whose_squares_vanish(monkeypatch):
    x, wg, bias, sel = draw(300, 512, 256, 12)
    x[100:] = 0  # a padded batch
    tiny = x.clone()
    tiny[:100] *= 2.0 ** -90
    zero = wg.clone()
    zero[::2] = 0
    for gate in (dict(), dict(n_group=8, topk_group=4), dict(score="softmax")):
        b = sel if not gate or "n_group" in gate else None
        for y in (x, tiny):
            for m in (wg, zero, wg * 0):
                check(monkeypatch, y, m, bias, b, 8, **gate)
                check(monkeypatch, y, m, None, b, 8, **gate)
        check(monkeypatch, tiny, wg * 2.0 ** -60, None, b, 8, full=None, **gate)  # products vanish too


def test_every_logit_formed_where_a_bound_is_missed(monkeypatch):
    x, wg, bias, sel = draw(1024, 512, 256, 10)
    monkeypatch.setenv("MOE_ROUTER_TC_BOUND", "-1")
    check(monkeypatch, x, wg, bias, sel, 8, full=None, n_group=8, topk_group=4)
    _, _, st = route(monkeypatch, True, x, wg, bias, sel, 8, dict(n_group=8, topk_group=4))
    assert st[1] == 1024


def test_captured_and_replayed(monkeypatch):
    t = torch()
    monkeypatch.setenv("MOE_ROUTER_TC_MIN_TOKENS", "1")
    x, wg, bias, sel = draw(1100, 512, 256, 11)
    s, gate = moe.shape_of(1100, 512, 256, 8, 128), moe.gate_of(n_group=8, topk_group=4)
    ws = t.empty(moe.moe_workspace_size(s), dtype=t.uint8, device="cuda")
    idx = t.empty(1100, 8, dtype=t.int32, device="cuda")
    w = t.empty(1100, 8, device="cuda")
    call = lambda i, v: moe.moe_route_gate(s, gate, x, wg, bias, sel, i, v, ws)
    stream = t.cuda.Stream()
    stream.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(stream):
        call(idx, w)
        graph = t.cuda.CUDAGraph()
        with t.cuda.graph(graph, stream=stream):
            call(idx, w)
    t.cuda.synchronize()
    x.copy_(x.flip(0))
    idx.fill_(-1)
    graph.replay()
    t.cuda.synchronize()
    i2, w2 = t.empty_like(idx), t.empty_like(w)
    call(i2, w2)
    t.cuda.synchronize()
    assert (idx == i2).all() and (w == w2).all()
