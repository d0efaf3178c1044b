"""Host-side checks of the attention entry points: every bad argument is refused before a launch,
so no GPU is needed."""
import ctypes

import pytest

import routed_expert_ffn_moe_gb300 as moe
from routed_expert_ffn_moe_gb300 import build as moe_build

F = 0x7F0000000000  # never dereferenced: every call below fails host validation
WS = 1 << 40


@pytest.fixture(scope="module", autouse=True)
def _lib():
    moe_build.build()
    moe.load()


def shape(**kw):
    base = dict(T=4, B=4, Hq=8, Hkv=2, D=128, page_size=16, max_pages=8, num_pages=64, rot_dim=128,
                max_pos=128)
    base.update(kw)
    return moe.attn_shape(**base)


BAD = [
    (dict(D=96), -2, "D=96"), (dict(Hq=9), -1, "Hq=9"), (dict(Hkv=0), -1, "Hkv=0"),
    (dict(Hq=129, Hkv=1), -1, "Hq=129"), (dict(T=-1), -1, "T=-1"), (dict(B=-1), -1, "B=-1"),
    (dict(page_size=0), -1, "page_size=0"), (dict(max_pages=0), -1, "max_pages=0"),
    (dict(num_pages=0), -1, "num_pages=0"),
    (dict(page_size=1 << 20, max_pages=1 << 20), -1, "2^30"),
    (dict(window=-1), -1, "window=-1"), (dict(n_sink=-1), -1, "n_sink=-1"),
    (dict(rot_dim=8), -1, "rot_dim=8"), (dict(rot_dim=144), -1, "rot_dim=144"),
    (dict(max_pos=-1), -1, "max_pos"), (dict(scale=-1.0), -1, "scale=-1"),
    (dict(scale=float("nan")), -1, "scale"), (dict(eps=float("inf")), -1, "eps"),
    (dict(kv_dtype=2), -1, "kv_dtype=2"),
    (dict(q_stride=8 * 128 + 4), -1, "q_stride"), (dict(q_stride=512), -1, "q_stride"),
    (dict(k_stride=-8), -1, "k_stride"), (dict(qr_stride=1), -1, "qr_stride"),
    (dict(o_stride=8), -1, "o_stride"), (dict(page_stride=1 << 20), -1, "together"),
    (dict(page_stride=8 * 4096, head_stride=2048, token_stride=132), -1, "token_stride"),
    (dict(page_stride=128, head_stride=2048, token_stride=128), -1, "page_stride"),
    (dict(kv_dtype="fp8", page_stride=1 << 20, head_stride=128 * 16, token_stride=136), -1,
     "token_stride"),
]


@pytest.mark.parametrize("kw,code,word", BAD, ids=[str(b[0]) for b in BAD])
def test_bad_shapes_are_refused(kw, code, word):
    s = shape(**kw)
    assert moe.moe_attn_workspace_size(s) == 0
    with pytest.raises(moe.MoeError) as ei:
        moe.moe_attn_decode(s, F, F, F, None, None, F, F, F, None, F, stream=0, ws_bytes=WS)
    assert ei.value.status == code and word in str(ei.value)
    with pytest.raises(moe.MoeError) as ei:
        moe.moe_attn_append(s, F, F, F, F, F, F, F, F, F, F, None, None, F, F, F, F, stream=0,
                            ws_bytes=WS)
    assert ei.value.status == code and word in str(ei.value)


def refused(fn, args, word, code=-1, ws=F, ws_bytes=WS, s=None):
    with pytest.raises(moe.MoeError) as ei:
        fn(s or shape(), *args, ws, stream=0, ws_bytes=ws_bytes)
    assert ei.value.status == code and word in str(ei.value), str(ei.value)


def test_bad_pointers_of_append_are_refused():
    # q, k, v, q_norm, k_norm, cos_sin, positions, table, kv_len, q_start, ks, vs, q_out, kc, vc
    good = [F, F, F, F, F, F, F, F, F, F, None, None, F + 64, F, F]
    for i, name in ((0, "q "), (1, "k "), (2, "v "), (5, "cos_sin"), (7, "block_table"),
                    (8, "kv_len"), (12, "q_out"), (13, "k_cache"), (14, "v_cache")):
        bad = list(good)
        bad[i] = None
        refused(moe.moe_attn_append, bad, name + ("is NULL" if name.endswith(" ") else " is NULL"))
    for i, name in ((0, "q not"), (3, "q_norm"), (4, "k_norm"), (12, "q_out"), (14, "v_cache")):
        bad = list(good)
        bad[i] = F + 8
        refused(moe.moe_attn_append, bad, name)
    for i in (6, 7, 8, 9):
        bad = list(good)
        bad[i] = F + 2
        refused(moe.moe_attn_append, bad, "4-byte")
    bad = list(good)
    bad[10] = F
    refused(moe.moe_attn_append, bad, "must be NULL for a bf16 cache")
    bad = list(good)
    bad[9] = None
    refused(moe.moe_attn_append, bad, "q_start", s=shape(T=5))
    bad = list(good)
    bad[12] = F
    refused(moe.moe_attn_append, bad, "q_out is q", s=shape(q_stride=4096))
    n = moe.moe_attn_workspace_size(shape())
    refused(moe.moe_attn_append, good, "workspace", code=-3, ws_bytes=n - 1)
    refused(moe.moe_attn_append, good, "ws not 256", ws=F + 16)


def test_bad_pointers_of_decode_are_refused():
    # q, k_cache, v_cache, k_scale, v_scale, table, kv_len, o, lse
    good = [F, F, F, None, None, F, F, F, F]
    for i, name in ((0, "q is NULL"), (1, "k_cache"), (2, "v_cache"), (5, "block_table"),
                    (6, "kv_len"), (7, "o is NULL")):
        bad = list(good)
        bad[i] = None
        refused(moe.moe_attn_decode, bad, name)
    for i, name in ((0, "q not"), (7, "o not")):
        bad = list(good)
        bad[i] = F + 8
        refused(moe.moe_attn_decode, bad, name)
    bad = list(good)
    bad[8] = F + 2
    refused(moe.moe_attn_decode, bad, "lse")
    bad = list(good)
    bad[3] = F
    refused(moe.moe_attn_decode, bad, "must be NULL for a bf16 cache")
    refused(moe.moe_attn_decode, good, "one token per sequence", s=shape(T=5))
    n = moe.moe_attn_workspace_size(shape())
    refused(moe.moe_attn_decode, good, "workspace", code=-3, ws_bytes=n - 1)
    refused(moe.moe_attn_decode, good, "ws is NULL", ws=None)
    assert moe.load().moe_attn_decode(None, *good[:1], F, F, None, None, F, F, F, F, F, WS,
                                      None) == -1
    assert "shape is NULL" in moe.moe_last_error_string()


def test_bad_pointers_of_prefill_are_refused():
    # q, k_cache, v_cache, k_scale, v_scale, table, kv_len, q_start, o, lse
    good = [F, F, F, None, None, F, F, F, F, F]
    for i, name in ((0, "q is NULL"), (1, "k_cache"), (2, "v_cache"), (5, "block_table"),
                    (6, "kv_len"), (7, "q_start"), (8, "o is NULL")):
        bad = list(good)
        bad[i] = None
        refused(moe.moe_attn_prefill, bad, name)
    for i, name in ((0, "q not"), (8, "o not")):
        bad = list(good)
        bad[i] = F + 8
        refused(moe.moe_attn_prefill, bad, name)
    bad = list(good)
    bad[9] = F + 2
    refused(moe.moe_attn_prefill, bad, "lse")
    bad = list(good)
    bad[4] = F
    refused(moe.moe_attn_prefill, bad, "must be NULL for a bf16 cache")
    refused(moe.moe_attn_prefill, good, "2^30", s=shape(T=1 << 24, Hkv=1024, Hq=1024))
    refused(moe.moe_attn_prefill, good, "D=32", code=-2, s=shape(D=32, rot_dim=0))
    # an E4M3 cache is unpacked first: the plain workspace is too small for that
    s = shape(kv_dtype="fp8")
    n = moe.moe_attn_workspace_size(s)
    assert moe.moe_attn_workspace_size(s, True) >= n + 4 * 4 * 2 * 8 * 16 * 128
    refused(moe.moe_attn_prefill, good, "workspace", code=-3, ws_bytes=n, s=s)


def test_empty_steps_launch_nothing():
    s = shape(T=0, B=0)
    moe.moe_attn_prefill(s, *[None] * 10, F, stream=0, ws_bytes=WS)
    moe.moe_attn_decode(s, None, None, None, None, None, None, None, None, None, F, stream=0,
                        ws_bytes=WS)
    moe.moe_attn_append(s, *[None] * 15, F, stream=0, ws_bytes=WS)


def test_workspace_sizes():
    n = moe.moe_attn_workspace_size(shape())
    assert n > moe.moe_attn_workspace_zero_bytes() >= 4 and n % 256 == 0
    # it does not grow with the batch or the cache
    assert moe.moe_attn_workspace_size(shape(T=4096, B=4096, max_pages=8192)) == n
    assert ctypes.sizeof(moe.MoeAttnShape) == 14 * 4 + 2 * 4 + 8 * 8
