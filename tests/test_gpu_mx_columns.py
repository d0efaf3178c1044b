"""The MXFP4 operators on columns of one buffer: other columns do not overlap and are taken, shared ones are refused."""
import pytest

import routed_expert_ffn_moe_gb300 as moe
from gpu_helpers import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from routed_expert_ffn_moe_gb300 import build
    build.build()
    moe.load()


@pytest.mark.parametrize("T", [1, 20, 140, 600])
def test_projection_between_columns_of_one_buffer(T):
    t = torch()
    g = t.Generator(device="cuda").manual_seed(T)
    K, N = 256, 136
    layer = moe.MxLinear.from_weight(t.randn(N, K, generator=g, device="cuda").to(t.bfloat16), max_tokens=600)
    buf = t.randn(T, 640, generator=g, device="cuda").to(t.bfloat16)
    x, r, y = buf[:, :K], buf[:, K:K + N], buf[:, 400:400 + N]
    ref = layer.forward(x.contiguous(), r.contiguous()).clone()
    before = buf.clone()
    assert layer.forward(x, r, y) is y and (y == ref).all()
    assert (buf[:, :400] == before[:, :400]).all() and (buf[:, 400 + N:] == before[:, 400 + N:]).all()
    assert (layer.forward(x, r, r) == ref).all()  # in place
    layer.check()
    for out in (buf[:, K - 8:K - 8 + N], buf[:, K + 8:K + 8 + N]):
        with pytest.raises(moe.MoeError, match="overlaps"):
            layer.forward(x, r if out.data_ptr() > r.data_ptr() else None, out)
    square = moe.MxLinear.from_weight(t.randn(K, K, generator=g, device="cuda").to(t.bfloat16), max_tokens=600)
    with pytest.raises(moe.MoeError):
        square.forward(square.forward(x))  # its own buffer, which this call would write


def test_rows_back_beside_other_columns():
    t = torch()
    x = t.randn(50, 96, device="cuda").to(t.bfloat16)
    r = moe.mx_rows(50, 96)
    codes = t.empty(50, 48, dtype=t.uint8, device="cuda")
    scales = t.empty(50, 3, dtype=t.uint8, device="cuda")
    moe.moe_mx_quantize(r, x, codes, scales)
    y = t.empty_like(x)
    moe.moe_mx_dequantize(r, codes, scales, y)
    buf = t.zeros(50, 200, dtype=t.bfloat16, device="cuda")
    buf[:, :96] = x
    apart = moe.mx_rows(50, 96, stride=200)
    c2, s2 = t.empty_like(codes), t.empty_like(scales)
    moe.moe_mx_quantize(apart, buf, c2, s2)
    assert (c2 == codes).all() and (s2 == scales).all()
    moe.moe_mx_dequantize(apart, codes, scales, buf[:, 104:])
    assert (buf[:, :96] == x).all() and (buf[:, 104:] == y).all() and (buf[:, 96:104] == 0).all()
