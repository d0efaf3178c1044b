"""Places beyond 32 bits, the longest rows, and the most tokens: sampled against the definitions."""
import numpy as np
import pytest

import routed_expert_ffn_moe_gb300 as moe
from gpu_helpers import torch
from mx_helpers import quantised, random_mx, selected, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from routed_expert_ffn_moe_gb300 import build
    build.build()
    moe.load()


def test_quantise_over_2_to_31_elements():
    t = torch()
    rows, K = 140_001, 16384  # 2.3e9 elements, a slab of rows and a rest
    x = t.empty(rows, K, dtype=t.bfloat16, device="cuda").normal_(generator=t.Generator(device="cuda").manual_seed(1))
    at = [0, 1, 65535, 65536, 65537, 131071, 131072, rows - 1]
    v, byte = quantised(x[at].double().cpu().numpy())
    for tiles in (False, True):
        r = moe.mx_rows(rows, K, tiles=tiles)
        codes = t.empty(rows, K // 2, dtype=t.uint8, device="cuda")
        scales = t.empty(moe.moe_mx_scale_bytes(r), dtype=t.uint8, device="cuda")
        moe.moe_mx_quantize(r, x, codes, scales)
        if not tiles:
            s = scales.view(rows, -1)[at]
            assert (s.cpu().numpy() == byte).all()
            assert (values(codes[at], s).cpu().numpy() == v).all()
        back = t.zeros_like(x)
        moe.moe_mx_dequantize(r, codes, scales, back)
        assert (back[at].double().cpu().numpy() == v).all()
        del back
    t.cuda.empty_cache()


@pytest.mark.parametrize("N", [32771, 32768])  # rows stored by words, and by tensor maps
def test_product_over_2_to_31_outputs(N):
    t = torch()
    T, K = 66_000, 64
    wc, wsc = random_mx(N, K, 2)
    r = moe.mx_rows(N, K, tiles=True)
    wt = t.empty(moe.moe_mx_scale_bytes(r), dtype=t.uint8, device="cuda")
    moe.moe_mx_tile_scales(r, wsc, wt)
    x = t.randn(T, K, generator=t.Generator(device="cuda").manual_seed(3), device="cuda", dtype=t.bfloat16)
    shape = moe.mx_shape(T, N, K)
    y = t.empty(T, N, dtype=t.bfloat16, device="cuda")
    ws = t.zeros(moe.moe_mx_linear_workspace_size(shape), dtype=t.uint8, device="cuda")
    moe.moe_mx_linear(shape, x, None, wc, wt, None, None, y, ws)
    moe.moe_check_device_status(ws)
    at = [0, 255, 256, 65500, 65535, 65536, T - 1]
    xv = t.from_numpy(quantised(x[at].double().cpu().numpy())[0]).cuda()
    wv = values(wc, wsc)
    ref = xv @ wv.T
    acc = (K + 2) * 2.0 ** -23 * (xv.abs() @ wv.abs().T)  # as in the other products' tests
    assert ((y[at].double() - ref).abs() <= acc + 2.0 ** -8 * (ref.abs() + acc) + 2.0 ** -133).all()
    del y
    t.cuda.empty_cache()


@pytest.mark.parametrize("T", [1, 30, 200])
def test_the_longest_rows(T):
    t = torch()
    N, K = 96, 1 << 17
    wc, wsc = random_mx(N, K, 4)
    r = moe.mx_rows(N, K, tiles=True)
    wt = t.empty(moe.moe_mx_scale_bytes(r), dtype=t.uint8, device="cuda")
    moe.moe_mx_tile_scales(r, wsc, wt)
    x = t.randn(T, K, generator=t.Generator(device="cuda").manual_seed(5), device="cuda", dtype=t.bfloat16)
    shape = moe.mx_shape(T, N, K)
    y = t.empty(T, N, dtype=t.bfloat16, device="cuda")
    ws = t.zeros(moe.moe_mx_linear_workspace_size(shape), dtype=t.uint8, device="cuda")
    moe.moe_mx_linear(shape, x, None, wc, wt, None, None, y, ws)
    moe.moe_check_device_status(ws)
    xv = t.from_numpy(quantised(x.double().cpu().numpy())[0]).cuda()
    wv = values(wc, wsc)
    ref = xv @ wv.T
    acc = (K + 2) * 2.0 ** -23 * (xv.abs() @ wv.abs().T)
    assert ((y.double() - ref).abs() <= acc + 2.0 ** -8 * (ref.abs() + acc)).all()
    # far below that bound, which is loose for so many terms: rounding to bf16 is the most of the error
    assert ((y.double() - ref).norm() / ref.norm()).item() < 2.0 ** -8


@pytest.mark.parametrize("E,kw", [(1024, dict(n_group=16, topk_group=4)), (256, dict(n_group=8, topk_group=4))])
def test_selection_over_2_to_31_logits(E, kw):
    t = torch()
    T, k = (1 << 31) // E + 3000, 8
    l = t.empty(T, E, device="cuda").normal_(generator=t.Generator(device="cuda").manual_seed(6))
    b = t.randn(E, generator=t.Generator(device="cuda").manual_seed(7), device="cuda") * 0.05
    idx = t.full((T, k), -7, dtype=t.int32, device="cuda")
    w = t.empty(T, k, device="cuda")
    moe.moe_route_select(moe.shape_of(T, 128, E, k, 128), moe.gate_of(**kw), l, b, idx, w)
    at = np.r_[0:50, T - 3050:T - 2950, T - 50:T]
    ri, rw = selected(l[at].cpu().numpy(), b.cpu().numpy(), k, **kw)
    np.testing.assert_array_equal(idx[at].cpu().numpy(), ri)
    assert np.abs(w[at].cpu().numpy() - rw).max() < 2.0 ** -17
    assert (idx >= 0).all() and (idx < E).all()
    del l, idx, w
    t.cuda.empty_cache()
