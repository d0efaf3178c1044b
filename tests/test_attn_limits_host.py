"""Sizes of the attention workspace at the far end of the shapes; no GPU needed."""
import pytest

import routed_expert_ffn_moe_gb300 as moe
from routed_expert_ffn_moe_gb300 import build as moe_build

F = 0x7F0000000000  # never dereferenced: the calls fail host validation


@pytest.fixture(scope="module", autouse=True)
def _lib():
    moe_build.build()
    moe.load()


@pytest.mark.parametrize("kw", [
    # 4 B Hkv places D bytes: 2^64 and more, which no size_t holds
    dict(B=1 << 20, Hkv=1024, page_size=1 << 20, max_pages=1 << 10, kv_dtype="fp8"),
    dict(B=1 << 18, Hkv=1024, page_size=1 << 20, max_pages=1 << 10, kv_dtype="fp8", D=64),
    dict(B=1 << 20, Hkv=512, page_size=(1 << 20) + 8, max_pages=1000),
    # and more than a tensor map's strides reach
    dict(B=1 << 10, Hkv=64, page_size=1 << 20, max_pages=64, kv_dtype="fp8"),
], ids=str)
def test_unpacked_rows_that_no_memory_holds_are_refused(kw):
    base = dict(T=8, Hq=kw["Hkv"], D=128, num_pages=1 << 10)
    s = moe.attn_shape(**{**base, **kw})
    assert moe.moe_attn_workspace_size(s, True) == 0
    assert "unpacked" in moe.moe_last_error_string()
    assert moe.moe_attn_workspace_size(s) > 0  # append and decode read the cache where it lies
    with pytest.raises(moe.MoeError) as ei:
        moe.moe_attn_prefill(s, F, F, F, None, None, F, F, F, F, None, F, stream=0, ws_bytes=1 << 62)
    assert ei.value.status == -1 and "unpacked" in str(ei.value)


def test_unpacked_rows_that_fit_are_sized_exactly():
    kw = dict(T=8, B=64, Hq=64, Hkv=8, D=128, page_size=16, max_pages=8192, num_pages=1 << 16)
    plain = moe.moe_attn_workspace_size(moe.attn_shape(**kw), True)
    fp8 = moe.moe_attn_workspace_size(moe.attn_shape(kv_dtype="fp8", **kw), True)
    assert fp8 - plain == 4 * 64 * 8 * 131072 * 128
