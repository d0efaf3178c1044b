"""The attention operators on the GPU against their definitions in 64 bits."""
import pytest
import torch

import routed_expert_ffn_moe_gb300 as moe
from attn_helpers import (F64, Step, check_attention, half_ulp_bf16, half_ulp_e4m3, norm64,
                          rotate64, workspace)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from routed_expert_ffn_moe_gb300 import build
    build.build()
    moe.load()


# ---- decode ----------------------------------------------------------------------------------

def run_decode(step, ws=None, **more):
    t, s = step.device(), step.shape(**more)
    ws = workspace(s) if ws is None else ws
    o = torch.full((step.T, step.Hq, step.D), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((step.T, step.Hq), float("nan"), device="cuda")
    moe.moe_attn_decode(s, t["q"], t["k"], t["v"], t["ks"], t["vs"], t["table"], t["lens"], o, lse,
                        ws)
    moe.moe_check_device_status(ws)
    return o, lse


LENS = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 1000]
DECODE = [
    dict(Hq=8, Hkv=1),
    dict(Hq=14, Hkv=2, page=64),                         # groups of 7
    dict(Hq=3, Hkv=3, page=1),                           # one query head a key head
    dict(Hq=40, Hkv=2, page=5, order="NHD"),             # groups of 20: two items a key head
    dict(Hq=128, Hkv=1, page=16),                        # the widest group
    dict(Hq=8, Hkv=2, D=64, page=100, order="gaps"),
    dict(Hq=16, Hkv=1, D=64),
    dict(Hq=14, Hkv=2, kv="fp8"),
    dict(Hq=32, Hkv=1, kv="fp8", page=7, order="NHD"),
    dict(Hq=6, Hkv=2, kv="fp8", D=64, page=32, order="gaps"),
    dict(Hq=4, Hkv=4, kv="fp8", scales=False),
    dict(Hq=8, Hkv=2, window=100),
    dict(Hq=8, Hkv=2, window=64, sink=4, page=8),
    dict(Hq=8, Hkv=2, window=1, sink=0),                 # only itself
    dict(Hq=8, Hkv=2, window=1, sink=70, kv="fp8"),
    dict(Hq=8, Hkv=2, window=128, sink=130, D=64),
    dict(Hq=8, Hkv=2, window=5000, sink=3),              # wider than every sequence
    dict(Hq=8, Hkv=2, spread=60.0),                      # sharp: one key takes nearly everything
    dict(Hq=8, Hkv=2, spread=0.0),                       # flat: every score is zero
]


@pytest.mark.parametrize("kw", DECODE, ids=[str(k) for k in DECODE])
def test_decode(kw):
    step = Step(lens=LENS, new=[1] * len(LENS), **kw)
    # pages that the window has left behind may be gone from the table
    if step.window:
        for b, n in enumerate(step.lens):
            for i in range(step.max_pages):
                j0, j1 = i * step.page, (i + 1) * step.page
                if j1 <= n - step.window and j0 >= step.sink:
                    step.table[b, i] = -1
    step2 = Step(lens=LENS, new=[1] * len(LENS), **kw)  # the reference keeps every page
    o, lse = run_decode(step)
    check_attention(step2, o, lse, str(kw))


@pytest.mark.parametrize("lens,kw", [
    ([1], dict(Hq=8, Hkv=1)),
    ([20011], dict(Hq=8, Hkv=1)),                                   # one sequence over every block
    ([9001, 3, 0, 777], dict(Hq=14, Hkv=2, kv="fp8", page=64)),
    (list(range(0, 90)) + [4000], dict(Hq=4, Hkv=2, D=64)),         # many short ones and a long one
    ([0] * 40, dict(Hq=4, Hkv=2)),
    ([33] * 700, dict(Hq=2, Hkv=1, D=64, page=32)),                 # more items than blocks
], ids=["one", "split", "fp8", "ragged", "empty", "items"])
def test_decode_splits(lens, kw):
    step = Step(lens=lens, new=[1] * len(lens), **kw)
    s = step.shape()
    ws = workspace(s)
    zero = moe.moe_attn_workspace_zero_bytes()
    first = run_decode(step, ws)
    check_attention(step, *first)
    assert not ws[:zero].any()  # left as it was found
    for _ in range(3):          # and the result does not depend on which block came last
        again = run_decode(step, ws)
        assert torch.equal(first[0].view(torch.int16), again[0].view(torch.int16))
        assert torch.equal(first[1], again[1])


def test_decode_without_lse_with_strides_and_scale_on_another_stream():
    step = Step(lens=[70, 5, 300], new=[1, 1, 1], Hq=8, Hkv=2)
    t = step.device()
    wide_q = torch.full((3, 8 * 128 + 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide_q[:, :8 * 128] = (step.q.cuda() * 2).view(3, -1)  # twice the queries at half the scale
    wide_o = torch.full((3, 8 * 128 + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    s = step.shape(qr_stride=8 * 128 + 64, o_stride=8 * 128 + 16, scale=0.5 / 128 ** 0.5)
    ws = workspace(s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    moe.moe_attn_decode(s, wide_q, t["k"], t["v"], None, None, t["table"], t["lens"], wide_o, None,
                        ws, stream=side)
    side.synchronize()
    ref, _, tol, _ = step.reference()
    o = wide_o[:, :8 * 128].reshape(3, 8, 128).cpu().to(F64)
    assert ((o - ref).abs() <= tol).all()
    assert (wide_o[:, 8 * 128:] == 7.0).all()  # nothing beyond the heads


def test_decode_records_bad_tables_and_lengths():
    step = Step(lens=[40, 40, 40], new=[1, 1, 1], Hq=4, Hkv=2)
    good = run_decode(step)
    t, s = step.device(), step.shape()
    for what in ("page", "negative", "length"):
        table, lens = t["table"].clone(), t["lens"].clone()
        if what == "length":
            lens[1] = 16 * step.max_pages + 1
        else:
            table[1, 1] = step.num_pages if what == "page" else -7
        ws, o = workspace(s), torch.zeros(3, 4, 128, dtype=torch.bfloat16, device="cuda")
        moe.moe_attn_decode(s, t["q"], t["k"], t["v"], None, None, table, lens, o, None, ws)
        with pytest.raises(moe.MoeError) as ei:
            moe.moe_check_device_status(ws)
        assert ei.value.status == -6
        moe.moe_check_device_status(ws)  # cleared by the read
        for b in (0, 2):                 # the other sequences are not disturbed
            assert torch.equal(o[b], good[0][b])


def test_decode_over_a_cache_past_32_bits():
    # 2^31 + 2^27 elements a cache (bf16: past 2^32 bytes), the sequence in its last pages
    Hkv, page, D = 8, 64, 128
    per = Hkv * page * D
    num = (2 ** 31 + 2 ** 27) // per
    n = 3 * page + 5
    small = Step(lens=[n], new=[1], Hq=16, Hkv=Hkv, page=page, extra_pages=0)
    caches = []
    for src in small.caches:
        big = torch.empty(num, Hkv, page, D, dtype=torch.bfloat16, device="cuda")
        big[-small.num_pages:] = src.cuda()
        caches.append(big)
    table = (small.table + (num - small.num_pages)).cuda()
    s = moe.attn_shape(T=1, B=1, Hq=16, Hkv=Hkv, D=D, page_size=page, max_pages=small.max_pages,
                       num_pages=num)
    ws = workspace(s)
    o = torch.empty(1, 16, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(1, 16, device="cuda")
    t = small.device()
    moe.moe_attn_decode(s, t["q"], *caches, None, None, table, t["lens"], o, lse, ws)
    moe.moe_check_device_status(ws)
    check_attention(small, o, lse)


# ---- append ----------------------------------------------------------------------------------

def append_case(lens, new, Hq, Hkv, D=128, kv="bf16", page=16, order="HND", rot=None, pairs=False,
                norm=True, positions=False, fused=True, in_place=False, null_start=False, seed=0,
                scales=True):
    rot = D if rot is None else rot
    step = Step(lens=lens, new=new, Hq=Hq, Hkv=Hkv, D=D, kv=kv, page=page, order=order, seed=seed,
                scales=scales)
    g = torch.Generator().manual_seed(seed + 1)
    T, nq, nk = step.T, Hq * D, Hkv * D
    qkv = (torch.randn(T, nq + 2 * nk, generator=g) * 3).to(torch.bfloat16)
    wq = (1 + 0.2 * torch.randn(D, generator=g)).to(torch.bfloat16) if norm else None
    wk = (1 + 0.2 * torch.randn(D, generator=g)).to(torch.bfloat16) if norm is True else None
    max_pos = max(max(lens), 1) + 50
    freq = 10000.0 ** (-torch.arange(rot // 2, dtype=F64) / max(rot // 2, 1))
    ang = torch.arange(max_pos, dtype=F64)[:, None] * freq
    cs = torch.cat([ang.cos(), ang.sin()], 1).float()
    t = step.device()
    place = torch.cat([torch.arange(n - m, n) for n, m in zip(lens, new)]) if T else torch.zeros(0)
    pos = place.long() + 37 if positions else place.long()

    dev = qkv.cuda()
    parts = [dev[:, :nq], dev[:, nq:nq + nk], dev[:, nq + nk:]]
    strides = dict(q_stride=nq + 2 * nk, k_stride=nq + 2 * nk, v_stride=nq + 2 * nk)
    if not fused:
        parts, strides = [p.contiguous() for p in parts], {}
    q_out = torch.full((T, Hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    if in_place:
        q_out = parts[0]
        strides["qr_stride"] = strides.get("q_stride", 0)
    s = step.shape(rot_dim=rot, rot_pairs=pairs, max_pos=max_pos, eps=1e-5, **strides)
    ws = workspace(s)
    before = [c.clone() for c in (t["k"], t["v"])]
    moe.moe_attn_append(s, *parts, wq.cuda() if norm else None, None if wk is None else wk.cuda(),
                        cs.cuda() if rot else None,
                        pos.to(torch.int32).cuda() if positions else None, t["table"], t["lens"],
                        None if null_start else t["q_start"], t["ks"], t["vs"], q_out, t["k"],
                        t["v"], ws)
    moe.moe_check_device_status(ws)

    # ---- the definition ----
    x = qkv.to(F64).view(T, Hq + 2 * Hkv, D)
    live = place >= 0
    c64, s64 = (cs.to(F64)[pos.clamp(0, max_pos - 1)][:, None, i * (rot // 2):(i + 1) * (rot // 2)]
                for i in range(2))
    q64 = rotate64(norm64(x[:, :Hq], wq, 1e-5), c64, s64, pairs)
    k64 = rotate64(norm64(x[:, Hq:Hq + Hkv], wk, 1e-5), c64, s64, pairs)
    q64[~live] = 0
    # fp32 arithmetic: the norm and the two products of a rotation are each within 2^-20 of the
    # head's largest element, then one rounding
    slack = lambda y: y.abs().amax(-1, keepdim=True) * 2.0 ** -19           # noqa: E731
    got = q_out.reshape(T, Hq, D).cpu().to(F64)
    assert ((got - q64).abs() <= half_ulp_bf16(q64) * 1.001 + slack(q64)).all()
    # caches: every place written, nothing else touched
    b_of = torch.repeat_interleave(torch.arange(step.B), torch.tensor(new))
    for name, y, sc, old in (("k", k64, step.k_scale, before[0]),
                             ("v", x[:, Hq + Hkv:], step.v_scale, before[1])):
        raw = t[name]
        touched = torch.zeros(raw.shape, dtype=torch.bool)
        tv = {"HND": lambda z: z, "NHD": lambda z: z.permute(0, 2, 1, 3),
              "gaps": lambda z: z[:step.num_pages, :Hkv, :page, :D]}[order]
        at = (step.table[b_of, (place.clamp(min=0) // page).long()].long()[live], slice(None),
              (place.clamp(min=0) % page).long()[live])
        tv(touched)[at] = True
        got = tv(raw.float().cpu())[at].to(F64)
        y = y[live]
        if kv == "fp8":
            y = y if sc is None else y / sc.to(F64)[:, None]
            tol = half_ulp_e4m3(y) * 1.001 + slack(y)
            y = y.clamp(-448, 448)
        else:
            tol = half_ulp_bf16(y) * 1.001 + slack(y)
            if name == "v":
                tol = torch.zeros_like(y)
        assert ((got - y).abs() <= tol).all(), name
        view = torch.int16 if kv == "bf16" else torch.uint8
        same = raw.view(view).cpu() == old.view(view).cpu()
        assert same[~touched].all(), name


@pytest.mark.parametrize("kw", [
    dict(lens=[1], new=[1], Hq=32, Hkv=8),
    dict(lens=[17, 1, 300, 64], new=[1] * 4, Hq=14, Hkv=2, null_start=True, in_place=True),
    dict(lens=[40, 5, 90, 7], new=[33, 5, 1, 0], Hq=8, Hkv=2, page=5, order="NHD"),
    dict(lens=[40, 5, 90, 7], new=[33, 5, 1, 0], Hq=8, Hkv=2, kv="fp8", page=7, order="gaps"),
    dict(lens=[129], new=[100], Hq=6, Hkv=3, D=64, pairs=True, rot=32, page=64),
    dict(lens=[129, 3], new=[100, 3], Hq=6, Hkv=3, D=64, rot=48, kv="fp8", scales=False),
    dict(lens=[129, 3], new=[100, 3], Hq=7, Hkv=1, rot=96, order="gaps", fused=False),
    dict(lens=[50], new=[50], Hq=128, Hkv=1, rot=16, pairs=True, fused=False, in_place=True),
    dict(lens=[50], new=[50], Hq=4, Hkv=4, rot=0, norm=False),
    dict(lens=[50, 60], new=[50, 2], Hq=4, Hkv=4, norm=False, positions=True),
    dict(lens=[0, 9, 0], new=[1, 1, 1], Hq=4, Hkv=2, null_start=True),      # padded batch
    dict(lens=[2, 9], new=[5, 1], Hq=4, Hkv=2),                             # three rows of padding
    dict(lens=[3] * 700, new=[1] * 700, Hq=4, Hkv=2, D=64),                 # more than a block's
    dict(lens=[3000], new=[2900], Hq=16, Hkv=8, kv="fp8", page=128),
    dict(lens=[30, 5], new=[30, 1], Hq=4, Hkv=4, norm="queries"),           # keys as they are
    # steps of more head rows than the small kernel takes, every kind of rotation
    dict(lens=[4000, 700, 3], new=[3900, 0, 3], Hq=14, Hkv=2, norm="queries"),
    dict(lens=[3000, 2500], new=[2000, 2500], Hq=7, Hkv=7, pairs=True, rot=64, order="NHD"),
    dict(lens=[1, 5000, 2], new=[3, 4000, 0], Hq=20, Hkv=1, kv="fp8", rot=48, page=7, order="gaps"),
    dict(lens=[6000], new=[5555], Hq=16, Hkv=2, D=64, page=100, in_place=True),
    dict(lens=[6000], new=[5555], Hq=16, Hkv=2, D=64, kv="fp8", rot=0, positions=True, norm=False),
], ids=lambda k: "-".join(f"{a}={b}" for a, b in k.items() if a not in ("lens", "new")))
def test_append(kw):
    append_case(**kw)


def test_append_skips_rows_after_the_last_sequence():
    step = Step(lens=[4, 6], new=[2, 3], Hq=4, Hkv=2)
    t = step.device()
    T = 9  # four rows of padding after the last sequence
    s = moe.attn_shape(T=T, B=2, Hq=4, Hkv=2, D=128, max_pages=step.max_pages,
                       num_pages=step.num_pages)
    x = torch.ones(T, 8 * 128, dtype=torch.bfloat16, device="cuda")
    q, k, v = x[:, :512].contiguous(), x[:, 512:768].contiguous(), x[:, 768:].contiguous()
    ws = workspace(s)
    out = torch.full((T, 4, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_attn_append(s, q, k, v, None, None, None, None, t["table"], t["lens"], t["q_start"],
                        None, None, out, t["k"], t["v"], ws)
    moe.moe_check_device_status(ws)
    assert (out[:5] == 1).all() and (out[5:] == 0).all()


@pytest.mark.parametrize("what", ["page", "length", "position"])
def test_append_records_what_is_out_of_range(what):
    step = Step(lens=[20, 20], new=[1, 1], Hq=4, Hkv=2)
    t = step.device()
    table, lens = t["table"].clone(), t["lens"].clone()
    max_pos = 64
    pos = torch.tensor([19, 19], dtype=torch.int32, device="cuda")
    if what == "page":
        table[0, 1] = step.num_pages
    elif what == "length":
        lens[0] = 16 * step.max_pages + 1
    else:
        pos[0] = max_pos
    s = step.shape(rot_dim=128, max_pos=max_pos)
    cs = torch.zeros(max_pos, 128, device="cuda")
    cs[:, :64] = 1
    k = torch.ones(2, 2, 128, dtype=torch.bfloat16, device="cuda")
    q = torch.ones(2, 4, 128, dtype=torch.bfloat16, device="cuda")
    out, ws = torch.empty_like(q), workspace(s)
    before = t["k"].clone()
    moe.moe_attn_append(s, q, k, k, None, None, cs, pos, table, lens, None, None, None, out,
                        t["k"], t["v"], ws)
    with pytest.raises(moe.MoeError) as ei:
        moe.moe_check_device_status(ws)
    assert ei.value.status == -6
    changed = (before.view(torch.int16) != t["k"].view(torch.int16)).any(-1).any(1)
    assert changed.sum().item() == 1  # only the other sequence's place was written
    assert (out[1] == 1).all()
