"""Prefill attention on the GPU against its definition in 64 bits."""
import pytest
import torch

import routed_expert_ffn_moe_gb300 as moe
from attn_helpers import F64, Step, check_attention, workspace

pytestmark = pytest.mark.gpu

# probabilities enter the product with v as bf16, eight significant bits
P_ROUND = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from routed_expert_ffn_moe_gb300 import build
    build.build()
    moe.load()


def run(step, ws=None, **more):
    t, s = step.device(), step.shape(**more)
    ws = workspace(s, True) if ws is None else ws
    o = torch.full((step.T, step.Hq, step.D), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((step.T, step.Hq), float("nan"), device="cuda")
    moe.moe_attn_prefill(s, t["q"], t["k"], t["v"], t["ks"], t["vs"], t["table"], t["lens"],
                         t["q_start"], o, lse, ws)
    moe.moe_check_device_status(ws)
    return o, lse


CASES = [
    dict(lens=[1], new=[1], Hq=8, Hkv=1),
    dict(lens=[37], new=[37], Hq=32, Hkv=8),
    dict(lens=[128], new=[128], Hq=2, Hkv=2),              # one full row tile, one key tile
    dict(lens=[300], new=[300], Hq=2, Hkv=2, page=128),    # both row tiles of a block
    dict(lens=[513, 0, 64, 129], new=[513, 0, 64, 129], Hq=14, Hkv=2, page=64),   # groups of 7
    dict(lens=[700, 40, 129], new=[3, 40, 1], Hq=8, Hkv=2),                       # over a cache
    dict(lens=[200, 200], new=[150, 10], Hq=6, Hkv=2, page=8),
    dict(lens=[260], new=[260], Hq=128, Hkv=1, page=256),                         # widest group
    dict(lens=[260], new=[260], Hq=100, Hkv=1),
    dict(lens=[260], new=[260], Hq=20, Hkv=1, order="NHD"),
    dict(lens=[260, 31], new=[260, 30], Hq=4, Hkv=2, order="gaps", page=32),
    dict(lens=[300, 70], new=[200, 70], Hq=8, Hkv=2, D=64),
    dict(lens=[300, 70], new=[200, 70], Hq=7, Hkv=1, D=64, page=128, order="NHD"),
    dict(lens=[300, 70], new=[200, 70], Hq=8, Hkv=2, page=5),                     # unpacked first
    dict(lens=[300, 70], new=[200, 70], Hq=8, Hkv=2, page=100, order="gaps"),
    dict(lens=[300, 70], new=[200, 70], Hq=8, Hkv=2, D=64, page=1),
    dict(lens=[300, 70, 1], new=[200, 70, 1], Hq=8, Hkv=2, kv="fp8"),
    dict(lens=[300, 70, 0], new=[200, 70, 0], Hq=8, Hkv=2, kv="fp8", D=64, page=7, order="NHD"),
    dict(lens=[300], new=[300], Hq=8, Hkv=2, kv="fp8", scales=False, page=64),
    dict(lens=[600], new=[600], Hq=8, Hkv=2, window=100),
    dict(lens=[600], new=[600], Hq=8, Hkv=2, window=128, sink=4),
    dict(lens=[900, 20], new=[100, 20], Hq=8, Hkv=2, window=200, sink=130),
    dict(lens=[900, 20], new=[100, 20], Hq=8, Hkv=2, window=1, sink=0),
    dict(lens=[900, 20], new=[300, 20], Hq=2, Hkv=2, window=1, sink=1, D=64),
    dict(lens=[900], new=[700], Hq=8, Hkv=2, window=256, sink=300, kv="fp8"),
    dict(lens=[600], new=[600], Hq=8, Hkv=2, window=5000, sink=7),
    dict(lens=[10, 300], new=[25, 280], Hq=8, Hkv=2),       # 15 rows of padding see nothing
    dict(lens=[10], new=[290], Hq=2, Hkv=2),                # a whole row tile of padding
    dict(lens=[300], new=[300], Hq=8, Hkv=2, spread=60.0),  # sharp
    dict(lens=[300], new=[300], Hq=8, Hkv=2, spread=0.0),   # flat
    dict(lens=[5] * 90 + [400], new=[5] * 90 + [333], Hq=4, Hkv=2),
    dict(lens=[3000], new=[1200], Hq=16, Hkv=2),            # the ring of tiles goes round
    dict(lens=[3000], new=[1200], Hq=16, Hkv=2, D=64, kv="fp8", page=64),
    # units that are cut along the keys: few rows over much, and more units than blocks
    dict(lens=[9000], new=[1], Hq=8, Hkv=1),
    dict(lens=[20011], new=[70], Hq=4, Hkv=1, page=64),
    dict(lens=[7000, 3, 5001, 0, 2500], new=[33, 3, 1, 0, 2500], Hq=14, Hkv=2),
    dict(lens=[9000, 8000], new=[5, 500], Hq=8, Hkv=2, D=64, page=32),
    dict(lens=[9000, 100], new=[400, 100], Hq=8, Hkv=2, window=3000, sink=200),
    dict(lens=[9000, 100], new=[400, 100], Hq=8, Hkv=2, D=64, window=1100, kv="fp8"),
    dict(lens=[6000], new=[2], Hq=2, Hkv=2, page=7),
    dict(lens=[1500] * 3, new=[1500] * 3, Hq=16, Hkv=2),
    dict(lens=[40] * 700, new=[1] * 700, Hq=2, Hkv=1),
    dict(lens=[70] * 300, new=[40] * 300, Hq=4, Hkv=2, D=64),
]


def forget(step):
    """Takes the pages from the table that no token of the step sees."""
    for b, (n, m) in enumerate(zip(step.lens, step.new)):
        for i in range(step.max_pages):
            j0, j1 = i * step.page, (i + 1) * step.page
            if step.window and j1 <= n - m - step.window + 1 and j0 >= step.sink:
                step.table[b, i] = -1


@pytest.mark.parametrize("kw", CASES, ids=[
    "-".join(f"{a}={b}" for a, b in k.items() if a not in ("lens", "new")) + f"-{i}"
    for i, k in enumerate(CASES)])
def test_prefill(kw):
    step, whole = Step(**kw), Step(**kw)
    forget(step)
    o, lse = run(step)
    check_attention(whole, o, lse, str(kw), P_ROUND)
    again = run(step)
    assert torch.equal(o.view(torch.int16), again[0].view(torch.int16))
    assert torch.equal(lse, again[1])


def test_split_rows_that_see_nothing_of_a_part():
    # a window that ends inside a part: some rows see nothing of the keys that a block walks, and
    # padding rows see nothing at all
    step = Step(lens=[6000, 30], new=[300, 40], Hq=2, Hkv=1, window=2000, sink=1500)
    o, lse = run(step)
    check_attention(step, o, lse, "parts", P_ROUND)


def test_rising_scores_raise_the_running_maximum():
    # keys that grow with their place: every tile's maximum is far above the one before
    step = Step(lens=[1500], new=[200], Hq=4, Hkv=1)
    grow = torch.linspace(0.1, 12, 1500)
    for i in range(step.max_pages):
        n = min(16, 1500 - 16 * i)
        page = step.k_view[int(step.table[0, i])]
        page[:, :n] = (grow[16 * i:16 * i + n, None] * torch.ones(128)).to(torch.bfloat16)
    step.q = torch.ones_like(step.q)
    o, lse = run(step)
    check_attention(step, o, lse, "rising", P_ROUND)


def test_strides_scale_and_another_stream():
    step = Step(lens=[70, 300], new=[70, 150], Hq=8, Hkv=2)
    t, T = step.device(), step.T
    wide_q = torch.full((T + 5, 8 * 128 + 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide_q[:T, :8 * 128] = (step.q.cuda() * 2).view(T, -1)
    wide_o = torch.full((T + 5, 8 * 128 + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    s = step.shape(qr_stride=8 * 128 + 64, o_stride=8 * 128 + 16, scale=0.5 / 128 ** 0.5)
    s.T = T + 5  # rows after the last sequence are padding
    ws = workspace(s, True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    moe.moe_attn_prefill(s, wide_q, t["k"], t["v"], None, None, t["table"], t["lens"],
                         t["q_start"], wide_o, None, ws, stream=side)
    side.synchronize()
    moe.moe_check_device_status(ws)
    ref, _, tol, _ = step.reference(P_ROUND)
    o = wide_o[:T, :8 * 128].reshape(T, 8, 128).cpu().to(F64)
    assert ((o - ref).abs() <= tol).all()
    assert (wide_o[:, 8 * 128:] == 7.0).all() and (wide_o[T:] == 7.0).all()


@pytest.mark.parametrize("kv,page", [("bf16", 16), ("bf16", 10), ("fp8", 16)])
def test_bad_tables_are_recorded(kv, page):
    step = Step(lens=[40, 40, 40], new=[40, 8, 40], Hq=4, Hkv=2, kv=kv, page=page)
    good = run(step)
    t, s = step.device(), step.shape()
    for what in ("page", "negative", "length"):
        table, lens = t["table"].clone(), t["lens"].clone()
        if what == "length":
            lens[1] = page * step.max_pages + 1
        else:
            table[1, 1] = step.num_pages if what == "page" else -7
        ws, o = workspace(s, True), torch.zeros(step.T, 4, 128, dtype=torch.bfloat16, device="cuda")
        moe.moe_attn_prefill(s, t["q"], t["k"], t["v"], t["ks"], t["vs"], table, lens,
                             t["q_start"], o, None, ws)
        with pytest.raises(moe.MoeError) as ei:
            moe.moe_check_device_status(ws)
        assert ei.value.status == -6
        for a, b in ((0, 40), (48, 88)):  # the other sequences are not disturbed
            assert torch.equal(o[a:b], good[0][a:b])


def test_one_token_a_sequence_agrees_with_decode():
    step = Step(lens=[5, 300, 129], new=[1, 1, 1], Hq=8, Hkv=2)
    o, lse = run(step)
    t, s = step.device(), step.shape()
    d_o, d_lse, ws = torch.empty_like(o), torch.empty_like(lse), workspace(s)
    moe.moe_attn_decode(s, t["q"], t["k"], t["v"], None, None, t["table"], t["lens"], d_o, d_lse, ws)
    _, _, tol, ltol = step.reference(P_ROUND)
    assert ((o.cpu().to(F64) - d_o.cpu().to(F64)).abs() <= 2 * tol).all()
    assert ((lse.cpu().to(F64) - d_lse.cpu().to(F64)).abs() <= 2 * ltol).all()


@pytest.mark.parametrize("D", [64, 128])
def test_every_tile_raises_the_maximum(D):
    """Keys that grow by more than the slack of the running maximum from tile to tile: every tile
    rescales the output, right behind the product of the tile before."""
    step = Step(lens=[4096, 700], new=[512, 700], Hq=8, Hkv=2, D=D, page=64)
    step.q = torch.ones_like(step.q)
    for b, n in enumerate(step.lens):
        for i in range(-(-n // 64)):
            m = min(64, n - 64 * i)
            # scores 16 i at the scale 1/sqrt(D): 2^23 from one tile to the next
            step.k_view[int(step.table[b, i])][:, :m] = 16 * i / D ** 0.5
    o, lse = run(step)
    check_attention(step, o, lse, "every tile", P_ROUND)
    for _ in range(20):
        again = run(step)
        assert torch.equal(o.view(torch.int16), again[0].view(torch.int16))
        assert torch.equal(lse, again[1])
