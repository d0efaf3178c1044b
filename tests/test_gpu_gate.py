"""Scored routing on the GPU against its formulas in 64 bits: every score, grouping and size, choices
nearer to each other than fp32 tells, masks, NaNs, other streams, graphs."""
import numpy as np
import pytest

import routed_expert_ffn_moe_gb300 as moe
from mx_helpers import selected
from gpu_helpers import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from routed_expert_ffn_moe_gb300 import build
    build.build()
    moe.load()


# Weights, relative: expf to 2 ulp (2^-22) of an argument rounded to 2^-24 of at most 20, twice (above
# and below the line), up to 69 roundings of a whole softmax's sum, division and scale: 119 * 2^-24.
W_REL = 2.0 ** -17


def run(logits, bias, k, **kw):
    t = torch()
    T, E = logits.shape
    idx = t.full((T, k), -7, dtype=t.int32, device="cuda")
    w = t.full((T, k), -7.0, device="cuda")
    s, g = moe.shape_of(T, 128, E, k, 128), moe.gate_of(**kw)
    moe.moe_route_select(s, g, t.as_tensor(logits, device="cuda"),
                         None if bias is None else t.as_tensor(bias, device="cuda"), idx, w)
    t.cuda.synchronize()
    return idx.cpu().numpy(), w.cpu().numpy()


def check(logits, bias, k, **kw):
    idx, w = run(logits, bias, k, **kw)
    ri, rw = selected(logits, bias, k, **kw)
    np.testing.assert_array_equal(idx, ri)
    np.testing.assert_array_equal(np.isnan(w), np.isnan(rw))
    ok = ~np.isnan(rw)
    assert (np.abs(w - rw)[ok] <= W_REL * np.abs(rw[ok]) + 1e-37).all()
    return idx, w


def draw(T, E, seed=0, spread=1.7):
    r = np.random.default_rng(seed)
    return (r.standard_normal((T, E)) * spread).astype(np.float32), (
        r.standard_normal(E) * 0.1).astype(np.float32)


GATES = [dict(n_group=1), dict(n_group=8, topk_group=4), dict(n_group=8, topk_group=3, group_top=1),
         dict(n_group=8, topk_group=8)]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("biased", [True, False])
@pytest.mark.parametrize("gate", GATES, ids=str)
def test_scores_groups_and_bias(score, biased, gate):
    l, b = draw(333, 256, 1)
    for renorm, scale in ((True, 2.5), (False, 1.0)):
        check(l, b if biased else None, 8, score=score, renorm=renorm, scale=scale, **gate)


# experts, groups, kept: quads and odd groups, groups of no power of two, the lanes' every share
SIZES = [(1, 1, 1), (2, 1, 1), (3, 3, 2), (8, 2, 1), (33, 1, 1), (60, 5, 3), (64, 32, 7), (66, 6, 2),
         (96, 3, 2), (160, 8, 3), (204, 17, 9), (264, 8, 5), (384, 1, 1), (511, 7, 3), (512, 16, 4),
         (1000, 1, 1), (1008, 28, 13), (1020, 17, 5), (1023, 31, 11), (1024, 1, 1), (1024, 32, 5)]


@pytest.mark.parametrize("E,G,keep", SIZES)
def test_sizes(E, G, keep):
    for T, k in ((1, 1), (7, 2), (9, 8), (33, 32)):
        k = min(k, keep * (E // G))
        l, b = draw(T, E, E + T)
        top = min(2, E // G)
        for bias in (b, None):
            check(l, bias, k, n_group=G, topk_group=keep, group_top=top)
        check(l, b, k, score="softmax", n_group=G, topk_group=keep, group_top=1, renorm=False)


def test_choices_nearer_than_fp32_tells():
    # biases that bring every c to within a rounding of one value: the order is in the 25th bit and beyond
    r = np.random.default_rng(5)
    for E, G, keep, k in ((256, 1, 1, 8), (64, 1, 1, 32), (256, 8, 4, 8), (40, 5, 2, 16), (384, 1, 1, 6)):
        for T in (1, 3):
            l = (r.standard_normal((1, E)) * 2).astype(np.float32).repeat(T, 0)
            b = (0.75 - 1 / (1 + np.exp(-l[0].astype(np.float64)))).astype(np.float32)
            check(l, b, k, n_group=G, topk_group=keep, scale=1.5)
    # two of many, at the border between chosen and not, in softmax as well
    for seed in range(20):
        l, b = draw(1, 128, 100 + seed)
        for score in ("sigmoid", "softmax"):
            s64 = selected(l, b, 9, score=score)[0][0]
            e, f = s64[7], s64[8]
            x = np.exp(l[0].astype(np.float64) - l.max())
            s = 1 / (1 + np.exp(-l[0].astype(np.float64))) if score == "sigmoid" else x / x.sum()
            b2 = b.copy()
            b2[f] = np.float32(s[e] + np.float64(b[e]) - s[f])
            check(l, b2, 8, score=score)


def test_exact_ties_go_to_the_lower_index():
    l, b = draw(64, 256, 7)
    l = np.round(l * 4) / 4  # few values, and so many equal logits
    for gate in GATES:
        check(l, None, 8, **gate)
        check(l, np.zeros(256, np.float32), 8, **gate)
    zero = np.zeros((5, 256), np.float32)
    for gate in GATES:
        idx, w = check(zero, None, 8, **gate)
        assert (idx == np.arange(8)).all() and np.allclose(w, 0.125)
        check(zero, np.zeros(256, np.float32), 8, score="softmax", **gate)


def test_masks_infinities_and_nans():
    l, b = draw(40, 256, 9)
    l[:, 100:] = -np.inf  # experts that are switched off
    l[3] = -np.inf        # a token without any
    l[4, :99] = -np.inf   # one expert left
    l[5, 17] = np.nan
    l[6] = np.nan
    l[7, 200] = np.inf
    l[8] = 60.0           # scores that round to 1 in 32 and 64 bits
    l[9] = -200.0         # scores that are 0 in 32 bits
    l[9, 5] = -199.0
    for gate in GATES[:2]:
        for bias in (None, b):
            check(l, bias, 8, **gate)
    off = b.copy()
    off[32:] = -np.inf  # whole groups switched off by the bias
    off[40] = np.nan
    for gate in GATES[:2]:
        check(draw(40, 256, 10)[0], off, 8, **gate)
    big = (b * 1e7).astype(np.float32)  # biases that leave few bits to the scores
    check(draw(40, 256, 11)[0], big, 8, n_group=8, topk_group=4)


def test_softmax_with_masked_logits():
    l, b = draw(16, 64, 12)
    l[:, 40:] = -np.inf
    check(l, None, 8, score="softmax")
    check(l, b, 8, score="softmax", renorm=False)
    check(l, None, 8, score="softmax", renorm=False, n_group=4, topk_group=2)


MANY = 6147  # tokens: eight lanes each, an odd number of them


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,G,keep,top,k", [
    (256, 8, 4, 2, 8), (256, 1, 1, 2, 8), (256, 8, 4, 1, 6), (384, 1, 1, 2, 6), (160, 8, 3, 1, 6), (64, 4, 1, 2, 3),
    (8, 1, 1, 2, 8), (8, 2, 1, 2, 4), (32, 8, 3, 2, 8), (16, 4, 2, 1, 1), (96, 3, 2, 2, 8), (100, 5, 2, 2, 7),
    (128, 2, 1, 2, 8), (336, 7, 3, 2, 8), (128, 1, 1, 2, 8), (320, 1, 1, 1, 4), (12, 1, 1, 2, 8)])
def test_many_tokens(E, G, keep, top, k, score):
    l, b = draw(MANY, E, E + k)
    for bias in (b, None):
        check(l, bias, k, score=score, n_group=G, topk_group=keep, group_top=top, renorm=k != 6, scale=1.5)


def test_many_tokens_ties_masks_and_near_choices():
    l, b = draw(MANY, 256, 21)
    l[:500] = np.round(l[:500] * 4) / 4
    l[500:700, 60:] = -np.inf
    l[700, 3] = np.nan
    l[701] = np.nan
    l[702, 77] = np.inf
    l[703] = -np.inf
    l[704] = 60.0
    l[705] = -200.0
    l[706] = 0
    l[707, 255] = 3e38
    l[708] *= 1e-42  # subnormal logits
    one = l[900].astype(np.float64)  # every c within a rounding of one value for these
    near = (0.75 - 1 / (1 + np.exp(-one))).astype(np.float32)
    l[901:950] = l[900]
    l[950:1000, 8:] = -30  # all eight from one lane's experts, or one group
    off = b.copy()
    off[200:] = -np.inf
    for gate in GATES:
        for bias in (None, b, near, off):
            check(l, bias, 8, **gate)


def test_a_token_by_itself_and_in_a_batch():
    l, b = draw(MANY, 256, 22)
    for kw in (dict(n_group=8, topk_group=4), dict(score="softmax")):
        idx, w = run(l, b, 8, **kw)
        i1, w1 = run(l[:7], b, 8, **kw)
        assert (idx[:7] == i1).all() and (w[:7].view(np.int32) == w1.view(np.int32)).all()


def test_neighbouring_memory_is_untouched():
    t = torch()
    l, b = draw(13, 60, 13)
    buf_i = t.full((13 * 6 + 64,), -9, dtype=t.int32, device="cuda")
    buf_w = t.full((13 * 6 + 64,), -9.0, device="cuda")
    moe.moe_route_select(moe.shape_of(13, 128, 60, 6, 128), moe.gate_of(), t.as_tensor(l).cuda(),
                         t.as_tensor(b).cuda(), buf_i, buf_w)
    assert (buf_i[13 * 6:] == -9).all() and (buf_w[13 * 6:] == -9).all()
    assert (buf_i[:13 * 6].view(13, 6).cpu().numpy() == selected(l, b, 6)[0]).all()


def test_another_stream_and_a_graph():
    t = torch()
    l, b = draw(300, 256, 14)
    lg, bg = t.as_tensor(l).cuda(), t.as_tensor(b).cuda()
    s, g = moe.shape_of(300, 128, 256, 8, 128), moe.gate_of(n_group=8, topk_group=4, scale=2.5)
    idx = t.empty(300, 8, dtype=t.int32, device="cuda")
    w = t.empty(300, 8, device="cuda")
    t.cuda.synchronize()
    st = t.cuda.Stream()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph, stream=st):
        moe.moe_route_select(s, g, lg, bg, idx, w)
    for seed in (15, 16):
        l2, _ = draw(300, 256, seed)
        lg.copy_(t.as_tensor(l2))
        graph.replay()
        t.cuda.synchronize()
        assert (idx.cpu().numpy() == selected(l2, b, 8, n_group=8, topk_group=4)[0]).all()
    with t.cuda.stream(st):
        moe.moe_route_select(s, g, lg, None, idx, w)
    st.synchronize()
    assert (idx.cpu().numpy() == selected(l2, None, 8, n_group=8, topk_group=4)[0]).all()


@pytest.mark.parametrize("T", [1, 5, 70, 1500])
def test_router_from_tokens(T):
    """moe_route_gate is moe_route's logits, then the selection: with softmax scores and no groups it gives
    moe_route's own choice, and with a gate that of moe_route_select on logits in 64 bits."""
    t = torch()
    d, E, k = 256, 128, 6
    g = t.Generator(device="cuda").manual_seed(T)
    x = t.randn(T, d, generator=g, device="cuda", dtype=t.bfloat16)
    wg = (t.randn(E, d, generator=g, device="cuda") * 0.1).to(t.bfloat16)
    bias = t.randn(E, generator=g, device="cuda") * 0.1
    sel = t.randn(E, generator=g, device="cuda") * 0.1
    s = moe.shape_of(T, d, E, k, 128)
    ws = t.full((moe.moe_workspace_size(s),), 255, dtype=t.uint8, device="cuda")
    out = [(t.empty(T, k, dtype=t.int32, device="cuda"), t.empty(T, k, device="cuda")) for _ in range(3)]
    moe.moe_route(s, x, wg, bias, *out[0], ws)
    moe.moe_check_device_status(ws)
    moe.moe_route_gate(s, moe.gate_of("softmax"), x, wg, bias, None, *out[1], ws)
    moe.moe_check_device_status(ws)
    assert (out[0][0] == out[1][0]).all()
    assert ((out[0][1] - out[1][1]).abs() <= 2 * W_REL * out[0][1]).all()
    gate = dict(n_group=8, topk_group=4, scale=2.5)
    moe.moe_route_gate(s, moe.gate_of(**gate), x, wg, bias, sel, *out[2], ws)
    logits = x.double() @ wg.double().T + bias.double()
    # fp32 sums of d products: d 2^-24 of their magnitudes, and the bias
    err = (x.double().abs() @ wg.double().abs().T + bias.abs()) * (d + 2) * 2.0 ** -24
    c = (logits.sigmoid() + sel.double()).cpu().numpy()
    ri, rw = selected(logits.cpu().numpy(), sel.cpu().numpy(), k, **gate)
    idx = out[2][0].cpu().numpy()
    same = (idx == ri).all(1)
    assert same.mean() > 0.99  # the others have neighbours within the logits' rounding
    e = err.max().item()
    for row in np.flatnonzero(~same):
        a, b = c[row, idx[row]], c[row, ri[row]]
        assert len(set(idx[row])) == k and (np.abs(np.sort(a) - np.sort(b)) <= 4 * e).all()
    assert np.abs(out[2][1].cpu().numpy() - rw)[same].max() <= 2.5 * (2 * e + W_REL)
