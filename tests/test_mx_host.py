"""Host-side checks of the MXFP4 operators: sizes, and every bad argument refused before a launch."""
import pytest

import routed_expert_ffn_moe_gb300 as moe
from routed_expert_ffn_moe_gb300 import build as moe_build

F = 0x7F0000000000  # never dereferenced: every call below fails host validation


@pytest.fixture(scope="module", autouse=True)
def _lib():
    moe_build.build()
    moe.load()


BAD_ROWS = [
    (dict(rows=-1), "rows=-1"), (dict(rows=(1 << 24) + 1), "rows"), (dict(K=0), "K=0"), (dict(K=48), "K=48"),
    (dict(K=(1 << 17) + 32), "K="), (dict(K=-32), "K=-32"), (dict(dtype=2), "dtype=2"), (dict(dtype=-1), "dtype=-1"),
    (dict(stride=32), "stride=32"), (dict(stride=68), "stride=68"), (dict(stride=-64), "stride=-64"),
    (dict(dtype="f32", stride=66), "stride=66"), (dict(stride=1 << 40), "stride"),
]


@pytest.mark.parametrize("kw,word", BAD_ROWS, ids=[str(b[0]) for b in BAD_ROWS])
def test_bad_rows_are_refused(kw, word):
    r = moe.mx_rows(**{**dict(rows=4, K=64), **kw})
    assert moe.moe_mx_scale_bytes(r) == 0
    for call in (moe.moe_mx_quantize, moe.moe_mx_dequantize):
        with pytest.raises(moe.MoeError) as ei:
            call(r, F, F + 512, F + 1024, stream=0)
        assert ei.value.status == -1 and word in str(ei.value)
    with pytest.raises(moe.MoeError):
        moe.moe_mx_tile_scales(r, F, F + 512, stream=0)


def test_sizes():
    assert moe.moe_mx_scale_bytes(moe.mx_rows(5, 96)) == 15
    assert moe.moe_mx_scale_bytes(moe.mx_rows(5, 96, tiles=True)) == 512
    assert moe.moe_mx_scale_bytes(moe.mx_rows(129, 160, tiles=True)) == 2 * 2 * 512
    # beyond 32 bits
    assert moe.moe_mx_scale_bytes(moe.mx_rows(1 << 24, 1 << 17, tiles=True)) == 1 << 36
    assert moe.moe_mx_linear_workspace_size(moe.mx_shape(0, 8, 32)) >= 256
    assert moe.moe_mx_linear_workspace_size(moe.mx_shape(100, 8, 64, "mxfp4")) >= 256
    assert moe.moe_mx_linear_workspace_size(moe.mx_shape(100, 8, 64)) >= 256 + 100 * 32 + 512


def test_quantise_pointers():
    r = moe.mx_rows(4, 64)
    for i, (a, b) in enumerate((("x", "codes"), ("codes", "scales"), ("scales", "y"))):
        for bad, says in ((None, "NULL"), (F + 8, "aligned")):
            args = [F, F + 512, F + 1024]
            args[i] = bad
            with pytest.raises(moe.MoeError, match=f"{a}.*{says}"):
                moe.moe_mx_quantize(r, *args, stream=0)
            with pytest.raises(moe.MoeError, match=f"{b}.*{says}"):
                moe.moe_mx_dequantize(r, *args, stream=0)
    with pytest.raises(moe.MoeError, match="same array"):
        moe.moe_mx_tile_scales(r, F, F, stream=0)
    for args in ((F, F, F + 512), (F, F + 512, F), (F, F + 512, F + 512)):
        with pytest.raises(moe.MoeError, match="of their own"):
            moe.moe_mx_quantize(r, *args, stream=0)
    for args in ((F, F + 512, F), (F, F + 512, F + 512)):
        with pytest.raises(moe.MoeError, match="of its own"):
            moe.moe_mx_dequantize(r, *args, stream=0)
    for call in (moe.moe_mx_quantize, moe.moe_mx_dequantize):  # no rows: no call
        call(moe.mx_rows(0, 64), None, None, None, stream=0)


BAD_SHAPES = [
    (dict(T=-1), "T=-1"), (dict(T=(1 << 24) + 1), "T="), (dict(N=0), "N=0"), (dict(N=(1 << 20) + 1), "N="),
    (dict(K=40), "K=40"), (dict(x_dtype=1), "x_dtype=1"), (dict(x_dtype=3), "x_dtype=3"),
    (dict(x_stride=56), "x_stride"), (dict(x_stride=68), "x_stride"), (dict(y_stride=7), "y_stride"),
    (dict(r_stride=7), "r_stride"), (dict(y_stride=-1), "y_stride"), (dict(x_dtype="mxfp4", x_stride=64), "x_stride"),
]


@pytest.mark.parametrize("kw,word", BAD_SHAPES, ids=[str(b[0]) for b in BAD_SHAPES])
def test_bad_shapes_are_refused(kw, word):
    s = moe.mx_shape(**{**dict(T=4, N=8, K=64), **kw})
    assert moe.moe_mx_linear_workspace_size(s) == 0
    with pytest.raises(moe.MoeError) as ei:
        moe.moe_mx_linear(s, F, F, F, F, None, None, F + 512, F, stream=0, ws_bytes=1 << 50)
    assert ei.value.status == -1 and word in str(ei.value)


def test_linear_pointers():
    for kind in ("bf16", "mxfp4"):
        s = moe.mx_shape(4, 8, 64, kind)
        n = moe.moe_mx_linear_workspace_size(s)
        good = [F, F if kind == "mxfp4" else None, F, F, None, None, F + 512, F]

        def refused(at, bad, status=-1, ws_bytes=n):
            args = list(good)
            args[at] = bad
            with pytest.raises(moe.MoeError) as ei:
                moe.moe_mx_linear(s, *args, stream=0, ws_bytes=ws_bytes)
            assert ei.value.status == status
            return str(ei.value)

        for at, name in ((0, "x "), (2, "w "), (3, "w_scales"), (6, "y "), (7, "ws ")):
            assert name + ("is NULL" if name[-1] == " " else " is NULL") in refused(at, None)
            assert "aligned" in refused(at, F + 8)
        assert "bias" in refused(4, F + 4) and "residual" in refused(5, F + 2)
        assert "workspace" in refused(0, F, -3, n - 1)
        assert "y is x or w" in refused(6, F)
        assert "x_scales" in refused(1, None if kind == "mxfp4" else F)
    s = moe.mx_shape(4, 8, 64, y_stride=16)
    with pytest.raises(moe.MoeError, match="residual is y"):
        moe.moe_mx_linear(s, F, None, F, F, None, F + 512, F + 512, F, stream=0, ws_bytes=1 << 20)
    moe.moe_mx_linear(moe.mx_shape(0, 8, 64), None, None, None, None, None, None, None, F, stream=0,
                      ws_bytes=1 << 20)
