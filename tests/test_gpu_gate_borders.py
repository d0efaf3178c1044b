"""Scored routing of large batches where eight lanes share a token: choices whose border runs through the experts
of one lane, nearer to each other than the keys tell, and groups by softmax scores of logits far from zero, against
the formulas in 64 bits."""
import numpy as np
import pytest

import routed_expert_ffn_moe_gb300 as moe
from gpu_helpers import torch
from test_gpu_gate import MANY, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from routed_expert_ffn_moe_gb300 import build
    build.build()
    moe.load()


def lane_experts(E, G):
    """Experts by lane: a group's quads of experts are dealt to the lanes of the group, 8 lanes a token."""
    lanes = 1
    while lanes < G:
        lanes *= 2
    P, per = 8 // lanes, E // G
    return [[g * per + e for e in range(per) if e // 4 % P == p] for g in range(G) for p in range(P)]


ULP = 2.0 ** -23


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("E,G,keep,top,k", [(256, 8, 2, 1, 8), (256, 1, 1, 2, 8), (256, 8, 8, 2, 8), (96, 1, 1, 2, 8),
                                            (384, 1, 1, 2, 8), (128, 2, 1, 1, 8), (256, 1, 1, 2, 7), (256, 8, 2, 1, 5)])
def test_a_border_within_a_lane(E, G, keep, top, k, biased):
    """A lane that gives up to eight of the k, and two to five more values that lie within the last bits of the k-th's
    key, its ninth and later ones among them; the rest of the k from other lanes."""
    r = np.random.default_rng(E + G + k)
    lanes = lane_experts(E, G)
    step = r.integers(0, 32, E) if not biased else r.integers(0, 5, E) * 13  # apart by more than the bounds of c
    l = np.empty((MANY, E), np.float32)
    for row in l:
        row[:] = r.uniform(-9, -4.5, E)
        lane = lanes[r.integers(len(lanes))]
        near = int(r.integers(2, 6))
        clear = int(r.integers(0, k))
        order = np.array(lane)[: clear + near] if r.random() < 0.5 else r.permutation(lane)[: clear + near]
        of_group = [e for e in range(E) if e // (E // G) == lane[0] // (E // G)]
        others = r.permutation([e for e in (range(E) if keep > 1 or G == 1 else of_group) if e not in lane])
        others = others[:max(0, k - clear - 1 - int(r.integers(0, 2)))]
        high = np.concatenate([order[:clear], others])
        row[high] = r.uniform(2, 12, len(high)) if not biased else r.uniform(0.5, 4, len(high))
        row[order[clear:]] = 1 + r.integers(0, 32, len(order) - clear) * ULP if not biased else 0.0
    bias = (0.5 + step * ULP).astype(np.float32) if biased else None
    check(l, bias, k, n_group=G, topk_group=keep, group_top=top)


def test_the_ninth_ends_a_lane():
    r = np.random.default_rng(3)
    l = r.standard_normal((MANY, 256)).astype(np.float32)
    rows = np.arange(5, MANY, 97)
    for row in rows:  # groups of 32 experts, one a lane: the ninth of the lane is the eighth of the token
        l[row] = r.uniform(-9, -4.5, 256)
        l[row, :6] = np.arange(10, 4, -1)
        l[row, [6, 7, 8]] = 1 + np.array([10, 5, 20]) * ULP
        l[row, 40] = 11
    idx, _ = check(l, None, 8, n_group=8, topk_group=2, group_top=1)
    assert (idx[rows] == [40, 0, 1, 2, 3, 4, 5, 8]).all()
    for row in rows:  # no groups
        l[row] = r.uniform(-9, -4.5, 256)
        l[row, [0, 1, 2, 3, 32, 33]] = np.arange(10, 4, -1)
        l[row, [34, 35, 64]] = 1 + np.array([10, 5, 20]) * ULP
        l[row, 4] = 11
    idx, _ = check(l, None, 8)
    assert (idx[rows] == [4, 0, 1, 2, 3, 32, 33, 64]).all()
    bias = np.full(256, 0.5, np.float32)  # c = sigmoid + bias, 0.5 and a bias of 0.5 and some steps
    bias[[34, 35, 64]] += (np.array([12, 0, 25]) * ULP).astype(np.float32)
    for row in rows:
        l[row] = r.uniform(-9, -4.5, 256)
        l[row, [0, 1, 2, 3, 32, 33]] = np.linspace(4, 2, 6)
        l[row, [34, 35, 64]] = 0
        l[row, 4] = 5
    idx, _ = check(l, bias, 8)
    assert (idx[rows] == [4, 0, 1, 2, 3, 32, 33, 64]).all()


@pytest.mark.parametrize("offset", [0.0, 4e4, -4e4, 1e5, 1e6, -1e6, 2.0 ** 21, 2.0 ** 22, -2.0 ** 22, 1e7])
@pytest.mark.parametrize("E,G,keep", [(64, 8, 1), (256, 8, 4), (384, 8, 3), (128, 4, 2), (160, 2, 1)])
def test_softmax_groups_far_from_zero(E, G, keep, offset):
    """Sums of two softmax scores make a group's value, whatever all logits have in common: groups whose best is
    the largest and whose second is low, against groups with two a little below."""
    r = np.random.default_rng(int(abs(offset)) % 1000 + E)
    per, T = E // G, 2050
    l = np.full((T, E), -1000.0)
    for g in range(G):
        at = np.argsort(r.random((T, per)), 1)[:, :2] + g * per
        alone = r.random(T) < 0.4
        first = np.where(alone, -r.choice([0.0, 0.25, 1.0], T), -r.choice([0.125, 0.25, 0.5, 0.75, 2.0, 15.0], T))
        second = np.where(alone, r.choice([-1.0, -2.0, -30.0], T), first - r.choice([0.125, 0.25, 1.0], T))
        np.put_along_axis(l, at, np.stack([first, second], 1), 1)
    l = (l + offset).astype(np.float32)
    check(l, None, 2, score="softmax", n_group=G, topk_group=keep)
    check(l, None, min(8, keep * per), score="softmax", n_group=G, topk_group=keep, renorm=False)


def test_softmax_group_values_of_large_logits():
    r = np.random.default_rng(11)
    l = (r.standard_normal((2048, 64)) * 2).astype(np.float32)
    rows = np.arange(3, 2048, 61)
    for X in (2.0 ** 21, 2.0 ** 22):
        for row in rows:
            l[row] = X - r.uniform(1000, 2000, 64)
            l[row, [0, 1, 8, 9]] = X - np.array([0, 2, 0.125 if X < 3e6 else 0.5, 0.25 if X < 3e6 else 0.5])
        idx, _ = check(l, None, 2, score="softmax", n_group=8, topk_group=1)
        assert (np.sort(idx[rows]) == [8, 9]).all()


@pytest.mark.parametrize("T", [1, 3, MANY])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,G,keep,k", [(16, 1, 1, 4), (64, 1, 1, 8), (64, 4, 2, 5), (256, 8, 4, 8), (384, 1, 1, 6),
                                        (1000, 1, 1, 8), (60, 5, 3, 32), (66, 6, 2, 7)])
def test_ties_at_the_border_and_values_near_them(E, G, keep, k, score, T):
    """Logits of few values, and biases that bring every c to within a rounding of one value: the k-th and the next
    are exact ties, and behind them experts whose c is larger in the 25th bit and beyond."""
    r = np.random.default_rng(E + k)
    for few in (2, 5, 12):
        l = (r.integers(0, few, (1, E)) * 0.375 - 1).astype(np.float32)
        x = l[0].astype(np.float64)
        s = 1 / (1 + np.exp(-x)) if score == "sigmoid" else np.exp(x - x.max()) / np.exp(x - x.max()).sum()
        b = (0.75 - s).astype(np.float32)
        check(l.repeat(T, 0), b, k, score=score, n_group=G, topk_group=keep)


@pytest.mark.parametrize("T", [5119, 5120, 5123])
def test_batches_around_the_one_that_settles(monkeypatch, T):
    """The batch from which only the needed logits are formed (512 x 256: 5120 tokens): the choice of all of them."""
    t = torch()
    g = t.Generator(device="cuda").manual_seed(T)
    x = t.randn(T, 512, generator=g, device="cuda", dtype=t.bfloat16)
    wg = (t.randn(256, 512, generator=g, device="cuda") * 0.1).to(t.bfloat16)
    sel = t.randn(256, generator=g, device="cuda") * 0.1
    s, gate = moe.shape_of(T, 512, 256, 8, 128), moe.gate_of(n_group=8, topk_group=4, scale=2.5)
    ws = t.full((moe.moe_workspace_size(s),), 255, dtype=t.uint8, device="cuda")
    out = []
    for least in (None, "1000000000"):  # the rule's own; every logit formed
        monkeypatch.delenv("MOE_ROUTER_TC_MIN_TOKENS", raising=False)
        if least:
            monkeypatch.setenv("MOE_ROUTER_TC_MIN_TOKENS", least)
        out.append((t.full((T, 8), -7, dtype=t.int32, device="cuda"), t.full((T, 8), -7.0, device="cuda")))
        moe.moe_route_gate(s, gate, x, wg, None, sel, *out[-1], ws)
        moe.moe_check_device_status(ws)
    assert (out[0][0] == out[1][0]).all() and (out[0][1] == out[1][1]).all()
