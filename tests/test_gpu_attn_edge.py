"""Attention on the GPU where a result could be lost: workspaces with what other calls left there,
rows whose scores are NaN, probabilities far below the largest, infinite elements, limits beyond
every place."""
import pytest
import torch

import routed_expert_ffn_moe_gb300 as moe
from attn_helpers import F64, Step, check_attention, workspace

pytestmark = pytest.mark.gpu

P_ROUND = 2.0 ** -8  # prefill: probabilities as one bf16 term


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from routed_expert_ffn_moe_gb300 import build
    build.build()
    moe.load()


def run_prefill(step, ws=None, **more):
    t, s = step.device(), step.shape(**more)
    ws = workspace(s, True) if ws is None else ws
    o = torch.full((step.T, step.Hq, step.D), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((step.T, step.Hq), float("nan"), device="cuda")
    moe.moe_attn_prefill(s, t["q"], t["k"], t["v"], t["ks"], t["vs"], t["table"], t["lens"],
                         t["q_start"], o, lse, ws)
    moe.moe_check_device_status(ws)
    return o, lse


def run_decode(step, ws=None, **more):
    t, s = step.device(), step.shape(**more)
    ws = workspace(s) if ws is None else ws
    o = torch.full((step.T, step.Hq, step.D), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((step.T, step.Hq), float("nan"), device="cuda")
    moe.moe_attn_decode(s, t["q"], t["k"], t["v"], t["ks"], t["vs"], t["table"], t["lens"], o, lse,
                        ws)
    moe.moe_check_device_status(ws)
    return o, lse


# ---- the workspace holds what other calls left there -------------------------------------------

LEFT = [
    # few rows over a middling length: less than a tile for each run of the grid
    dict(lens=[1100], new=[1], Hq=8, Hkv=1),
    dict(lens=[1100], new=[1], Hq=8, Hkv=1, D=64),
    dict(lens=[4000], new=[2], Hq=8, Hkv=1),
    dict(lens=[9000], new=[3], Hq=4, Hkv=1, D=64),
    dict(lens=[2000, 1500], new=[1, 40], Hq=2, Hkv=1, D=64, page=64),
    dict(lens=[2000], new=[1], Hq=8, Hkv=1, D=64, kv="fp8"),
    dict(lens=[3000], new=[5], Hq=8, Hkv=1, D=64, window=1500, sink=100),
    dict(lens=[20011], new=[70], Hq=4, Hkv=1),
    # unpacked first, parts of the rows not needed
    dict(lens=[300, 0, 900, 70], new=[20, 0, 100, 70], Hq=4, Hkv=2, kv="fp8", page=7, window=60, sink=9),
    dict(lens=[300, 900], new=[200, 3], Hq=4, Hkv=2, D=64, page=24, window=200, sink=130),
]


@pytest.mark.parametrize("kw", LEFT, ids=str)
@pytest.mark.parametrize("left", [float("nan"), 3.0])
def test_prefill_takes_nothing_from_the_workspace(kw, left):
    step = Step(**kw)
    s = step.shape()
    ws = workspace(s, True)
    ws[moe.moe_attn_workspace_zero_bytes():].view(torch.float32).fill_(left)
    o, lse = run_prefill(step, ws)
    check_attention(step, o, lse, str(kw), P_ROUND)


@pytest.mark.parametrize("kw", LEFT, ids=str)
@pytest.mark.parametrize("left", [float("nan"), 3.0])
def test_decode_takes_nothing_from_the_workspace(kw, left):
    step = Step(**dict(kw, new=[1] * len(kw["lens"])))
    s = step.shape()
    ws = workspace(s)
    ws[moe.moe_attn_workspace_zero_bytes():].view(torch.float32).fill_(left)
    o, lse = run_decode(step, ws)
    check_attention(step, o, lse, str(kw))


# ---- NaN scores -------------------------------------------------------------------------------

def put_key(step, b, j, value):
    """Sets the key of place j of sequence b (all heads)."""
    step.k_view[int(step.table[b, j // step.page]), :, j % step.page] = torch.full(
        (step.Hkv, step.D), value).to(step.k_view.dtype)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("what", ["decode", "prefill"])
def test_nan_in_a_query_makes_its_row_nan_and_no_other(what, D, kv):
    run = run_decode if what == "decode" else run_prefill
    kw = dict(lens=[1, 40, 300, 20011], new=[1, 1, 1, 1], Hq=40, Hkv=2, D=D, kv=kv)
    good = run(Step(**kw))
    step = Step(**kw)
    hit = torch.zeros(step.T, step.Hq, dtype=torch.bool)
    for b, h, d in ((0, 3, 0), (1, 0, D - 1), (2, 39, 17), (3, 21, 5), (3, 2, 40)):
        step.q[b, h, d] = float("nan")
        hit[b, h] = True
    o, lse = (x.cpu() for x in run(step))
    assert torch.isnan(o[hit]).all() and torch.isnan(lse[hit]).all()
    assert torch.equal(o[~hit].view(torch.int16), good[0].cpu()[~hit].view(torch.int16))
    assert torch.equal(lse[~hit], good[1].cpu()[~hit])


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("what", ["decode", "prefill"])
def test_nan_keys_make_their_sequence_nan(what, kv):
    """One place, every place, and every place of a block's part."""
    run = run_decode if what == "decode" else run_prefill
    kw = dict(lens=[1, 70, 9000, 9000, 33], new=[1] * 5, Hq=8, Hkv=1, kv=kv)
    good = run(Step(**kw))
    step = Step(**kw)
    for b, places in ((0, [0]), (1, range(70)), (2, range(4000, 5200)), (3, [8999])):
        for j in places:
            put_key(step, b, j, float("nan"))
    o, lse = (x.cpu() for x in run(step))
    assert torch.isnan(o[:4]).all() and torch.isnan(lse[:4]).all()
    assert torch.equal(o[4].view(torch.int16), good[0][4].cpu().view(torch.int16))
    assert torch.equal(lse[4], good[1][4].cpu())


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_scores_of_minus_infinity_count_as_not_seen(kv):
    """softmax of -inf scores is 0 each, and a row of nothing else has no sum: o = 0, lse = -inf."""
    step = Step(lens=[50, 50], new=[1, 1], Hq=4, Hkv=1, kv=kv, scales=False)
    for j in range(50):
        put_key(step, 0, j, 1.0)
    step.q[0] = -float("inf")
    o, lse = (x.cpu() for x in run_decode(step))
    assert (o[0] == 0).all() and torch.isinf(lse[0]).all() and (lse[0] < 0).all()
    assert torch.isfinite(o[1]).all()


# ---- probabilities far below the largest --------------------------------------------------------

@pytest.mark.parametrize("lens,D", [([600], 128), ([600], 64), ([20000], 128)])
@pytest.mark.parametrize("below", [10, 14, 18, 22, 26, 30, 36])
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_decode_keeps_small_probabilities(kv, below, lens, D):
    """One key whose value is zero takes nearly all of the softmax; the output is what the others add,
    each about 2^-below of it. Over E4M3 a probability is an f16 times 2^14: half its smallest step is
    2^-39 of the largest probability, for each of the n keys, beside the relative bound."""
    step = Step(lens=lens, new=[1], Hq=8, Hkv=1, D=D, kv=kv, scales=False, page=32)
    step.q = torch.full_like(step.q, 1.0)
    n = lens[0]
    big = below * 0.6931471805599453 / D ** 0.5  # times 1: every element of the key, score * scale
    for i in range(step.max_pages):
        m = min(32, n - 32 * i)
        page = int(step.table[0, i])
        step.k_view[page][:, :m] = torch.zeros(m, D).to(step.k_view.dtype)
        v = 1 + 0.25 * torch.arange(D) / D
        step.v_view[page][:, :m] = v.expand(1, m, D).to(step.v_view.dtype)
    put_key(step, 0, n // 2, big)
    at = int(step.table[0, (n // 2) // 32])
    step.v_view[at][:, (n // 2) % 32] = torch.zeros(D).to(step.v_view.dtype)
    o, lse = run_decode(step)
    ref, ref_lse, o_tol, lse_tol = step.reference()
    if kv == "fp8":
        o_tol = o_tol + n * 2.0 ** -39 * 1.25
    assert ((o.cpu().to(F64) - ref).abs() <= o_tol).all()
    assert ((lse.cpu().to(F64) - ref_lse).abs() <= lse_tol).all()


# ---- append: what does not turn is copied -------------------------------------------------------

@pytest.mark.parametrize("T", [3, 5000])     # the small kernel, the large one
@pytest.mark.parametrize("rot,pairs", [(0, False), (32, False), (32, True)])
@pytest.mark.parametrize("D,kv", [(128, "bf16"), (64, "bf16"), (128, "fp8")])
def test_append_copies_what_does_not_turn(D, kv, rot, pairs, T):
    """Heads without a norm: elements past rot_dim come out as they went in, infinities, NaN and negative
    zeros among them, and do not touch their neighbours."""
    Hq, Hkv = 6, 2
    step = Step(lens=[T], new=[T], Hq=Hq, Hkv=Hkv, D=D, kv=kv, scales=False)
    t = step.device()
    g = torch.Generator().manual_seed(5)
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g).to(torch.bfloat16)
    odd = torch.tensor([float("inf"), -float("inf"), float("nan"), -0.0, 3e38]).to(torch.bfloat16)
    for n in range(40):
        h = int(torch.randint(Hq + 2 * Hkv, (1,), generator=g))
        d = int(torch.randint(rot, D, (1,), generator=g))
        qkv[int(torch.randint(T, (1,), generator=g)), h, d] = odd[n % 5]
    ang = torch.rand(T, max(rot // 2, 1), generator=g) * 6
    cs = torch.cat([ang.cos(), ang.sin()], 1)
    row = (Hq + 2 * Hkv) * D
    s = step.shape(rot_dim=rot, rot_pairs=pairs, max_pos=T, q_stride=row, k_stride=row, v_stride=row)
    dev, ws = qkv.cuda().view(T, row), workspace(s)
    out = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    moe.moe_attn_append(s, dev, dev[:, Hq * D:], dev[:, (Hq + Hkv) * D:], None, None,
                        cs.cuda() if rot else None, None, t["table"], t["lens"], t["q_start"], None,
                        None, out, t["k"], t["v"], ws)
    moe.moe_check_device_status(ws)

    def same(a, b):
        nan = torch.isnan(a.float())
        assert torch.equal(nan, torch.isnan(b.float()))
        a, b = a.masked_fill(nan, 0), b.masked_fill(nan, 0)
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))

    same(out.cpu()[..., rot:], qkv[:, :Hq, rot:])
    j = torch.arange(T)
    for name, h0, e0 in (("k", Hq, rot), ("v", Hq + Hkv, 0)):
        got = t[name].float().cpu()[step.table[0, j // step.page].long(), :, j % step.page]
        want = qkv[:, h0:h0 + Hkv]
        if kv == "fp8":  # saturating
            want = want.float().clamp(-448, 448).to(torch.float8_e4m3fn).float().to(torch.bfloat16)
        same(got.to(torch.bfloat16)[..., e0:], want[..., e0:])
    assert torch.isfinite(out[..., :rot]).all()


# ---- limits beyond every place ------------------------------------------------------------------

MOST = 2 ** 31 - 1


@pytest.mark.parametrize("more", [
    dict(window=MOST, n_sink=0),
    dict(window=MOST, n_sink=MOST),
    dict(window=64, n_sink=MOST),
    dict(window=MOST - 40, n_sink=3),
], ids=["window", "both", "sinks", "nearly"])
@pytest.mark.parametrize("kw", [
    dict(lens=[10, 300, 700], new=[25, 280, 3], Hq=8, Hkv=2),             # 15 rows of padding
    dict(lens=[10, 300, 700], new=[25, 280, 3], Hq=8, Hkv=2, D=64, kv="fp8", page=24),
    dict(lens=[4000], new=[200], Hq=8, Hkv=2, page=64),
], ids=["bf16", "fp8", "long"])
def test_limits_beyond_every_place_are_none(kw, more):
    plain, step = Step(**kw), Step(**kw)
    o, lse = run_prefill(step, **more)
    check_attention(plain, o, lse, "prefill", P_ROUND)
    one = dict(kw, new=[1] * len(kw["lens"]))
    o, lse = run_decode(Step(**one), **more)
    check_attention(Step(**one), o, lse, "decode")
