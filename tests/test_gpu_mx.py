"""The MXFP4 operators on the GPU against 64-bit definitions: quantisation and back (exact), the product at
sizes around its tiles, splits and strides."""
import numpy as np
import pytest

import routed_expert_ffn_moe_gb300 as moe
import synth
from mx_helpers import quantised, random_mx, tile_index, values
from gpu_helpers import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from routed_expert_ffn_moe_gb300 import build
    build.build()
    moe.load()


# ---- quantisation --------------------------------------------------------------------------------

def sample(rows, K, kind, seed=0):
    t = torch()
    g = t.Generator().manual_seed(seed)
    x = t.randn(rows, K, generator=g) * t.exp2(t.randint(-9, 10, (rows, K // 32), generator=g).float()
                                               ).repeat_interleave(32, 1)
    x[t.rand(rows, K, generator=g) < 0.05] = 0
    return x.to(t.bfloat16 if kind == "bf16" else t.float32)


def quantise(x, tiles=False, stride=0, fill=77):
    t = torch()
    rows, K = x.shape
    r = moe.mx_rows(rows, K, "bf16" if x.dtype == t.bfloat16 else "f32", tiles, stride)
    codes = t.full((rows, K // 2), fill, dtype=t.uint8, device="cuda")
    scales = t.full((moe.moe_mx_scale_bytes(r),), fill, dtype=t.uint8, device="cuda")
    moe.moe_mx_quantize(r, x, codes, scales)
    return codes, scales


def back(codes, scales, kind, tiles=False, stride=0):
    t = torch()
    rows, K = codes.shape[0], 2 * codes.shape[1]
    dt = t.bfloat16 if kind == "bf16" else t.float32
    y = t.full((rows, max(stride, K)), 5.0, dtype=dt, device="cuda")
    moe.moe_mx_dequantize(moe.mx_rows(rows, K, kind, tiles, stride), codes, scales, y)
    assert (y[:, K:] == 5).all()
    return y[:, :K]


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 64), (1, 7168), (33, 96), (130, 160), (257, 2080), (40, 1024)])
@pytest.mark.parametrize("tiles", [False, True])
def test_there_and_back(rows, K, kind, tiles):
    x = sample(rows, K, kind, rows + K)
    codes, scales = quantise(x.cuda(), tiles)
    v, byte = quantised(x.double().numpy())
    if tiles:
        at, size = tile_index(rows, K)
        s = scales.cpu().numpy()
        assert s.size == size and (s[at] == byte).all()
        for j in range(K // 32, -(-K // 128) * 4):  # the last chunk's padding
            last = at[:, (j // 4) * 4 if j // 4 * 4 < K // 32 else 0] // 4 * 4 + j % 4
            assert (s[last] == 127).all()
    else:
        assert (scales.view(rows, -1).cpu().numpy() == byte).all()
        assert (values(codes, scales.view(rows, -1)).cpu().numpy() == v).all()
    for out in ("bf16", "f32"):
        assert (back(codes, scales, out, tiles).double().cpu().numpy() == v).all()


def test_rows_apart():
    t = torch()
    for kind, pad in (("bf16", 8), ("f32", 4), ("bf16", 40)):
        x = sample(50, 96 + pad, kind, pad) if (96 + pad) % 32 == 0 else t.cat(
            [sample(50, 96, kind, pad), t.full((50, pad), 1e9).to(t.bfloat16 if kind == "bf16" else t.float32)], 1)
        x = x.cuda()
        codes, scales = quantise(x[:, :96], stride=96 + pad)
        v, _ = quantised(x[:, :96].double().cpu().numpy())
        assert (back(codes, scales, kind, stride=96 + pad).double().cpu().numpy() == v).all()


def test_every_rounding_and_tie():
    """Every E2M1 value, every middle between two and the fp32 numbers next to it, in blocks whose largest element
    is 4, 6 or 7.99, at the smallest and the largest scales."""
    t = torch()
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    v = np.concatenate([[0, 0.5, 1, 1.5, 2, 3], mids, np.nextafter(np.float32(mids), np.float32(0)),
                        np.nextafter(np.float32(mids), np.float32(9))]).astype(np.float32)
    v = v[v <= 4][:30]
    rows = []
    for top in (4.0, 6.0, 7.99):
        for e in (-127, -126, -20, 0, 30, 124, 125):
            for sign in (1, -1):
                x = np.zeros(32, np.float32)
                with np.errstate(over="ignore", under="ignore"):
                    x[:len(v)] = np.ldexp(v * sign, e)
                    x[31] = np.ldexp(np.float32(top), e)
                rows.append(x)
    x = np.stack(rows)
    x = x[np.isfinite(x).all(1)]
    codes, scales = quantise(t.as_tensor(x).cuda())
    ref, byte = quantised(x)
    assert (scales.cpu().numpy() == byte[:, 0]).all()
    assert (values(codes, scales.view(-1, 1)).cpu().numpy() == ref).all()
    assert (back(codes, scales, "f32").double().cpu().numpy() == ref).all()


def test_zeros_infinities_and_nans():
    t = torch()
    x = sample(6, 96, "f32", 3)
    x[0] = 0
    x[1, 5] = float("nan")
    x[2, 40] = float("inf")
    x[3, 95] = -float("inf")
    x[4, 32:64] = 1e-45
    x[5, 0:32] = -0.0
    for kind in ("f32", "bf16"):
        y = x.to(t.bfloat16 if kind == "bf16" else t.float32)
        for tiles in (False, True):
            codes, scales = quantise(y.cuda(), tiles)
            v, byte = quantised(y.double().numpy())
            np.testing.assert_array_equal(back(codes, scales, kind, tiles).double().cpu().numpy(), v)
            if not tiles:
                assert (scales.view(6, 3).cpu().numpy() == byte).all()
                assert byte[0].tolist() == [127] * 3 and byte[1, 0] == byte[2, 1] == byte[3, 2] == 255


def test_same_codes_as_the_weight_generator():
    t = torch()
    cfg = synth.get_config("tiny", wdtype="mxfp4")
    bits = synth.host_w13_expert(cfg, 1)
    q, s = synth.quantize_mxfp4(bits)
    x = t.from_numpy(bits.view(np.int16)).view(t.bfloat16).cuda()
    codes, scales = quantise(x)
    assert (scales.view(x.shape[0], -1).cpu().numpy() == s).all()
    assert (values(codes, scales.view(x.shape[0], -1)) == values(t.from_numpy(q).cuda(), t.from_numpy(s).cuda())).all()


@pytest.mark.parametrize("rows,K", [(1, 32), (128, 128), (130, 160), (300, 7168)])
def test_tile_scales(rows, K):
    t = torch()
    s = t.randint(0, 256, (rows, K // 32), dtype=t.uint8, generator=t.Generator().manual_seed(1))
    r = moe.mx_rows(rows, K, tiles=True)
    tiles = t.full((moe.moe_mx_scale_bytes(r),), 3, dtype=t.uint8, device="cuda")
    moe.moe_mx_tile_scales(r, s.cuda(), tiles)
    at, size = tile_index(rows, K)
    got = tiles.cpu().numpy()
    assert got.size == size and (got[at] == s.numpy()).all()
    if K % 128:
        assert (got[at[:, -1] + 1] == 127).all()


# ---- product -------------------------------------------------------------------------------------

def tiled(scales):
    t = torch()
    r = moe.mx_rows(scales.shape[0], 32 * scales.shape[1], tiles=True)
    out = t.full((moe.moe_mx_scale_bytes(r),), 255, dtype=t.uint8, device="cuda")  # padding rows: NaN scales
    moe.moe_mx_tile_scales(r, scales, out)
    return out


def workspace(shape, fill=255):
    t = torch()
    ws = t.full((moe.moe_mx_linear_workspace_size(shape),), fill, dtype=t.uint8, device="cuda")
    ws[:4] = 0
    return ws


def bound(x, w, ref, bias, residual):
    """Largest error of an element: K products, a bias and a residual added in fp32, each addition off by at
    most 2^-23 of the magnitudes (the tensor cores may cut instead of rounding), then half a step of bf16."""
    mag = x.abs() @ w.abs().T
    if bias is not None:
        mag = mag + bias.double().abs()
    if residual is not None:
        mag = mag + residual.double().abs()
    acc = (x.shape[1] + 2) * 2.0 ** -23 * mag
    return acc + 2.0 ** -8 * (ref.abs() + acc) + 2.0 ** -133


def product(T, N, K, kind="bf16", bias=False, residual=False, seed=0, xs=0, ys=0, rs=0, alias=False):
    t = torch()
    g = t.Generator(device="cuda").manual_seed(seed)
    wc, wsc = random_mx(N, K, seed)
    if kind == "bf16":
        buf = t.full((T, max(xs, K)), float("nan"), dtype=t.bfloat16, device="cuda")
        x = buf[:, :K]
        x.copy_(t.randn(T, K, generator=g, device="cuda"))
        xv = t.from_numpy(quantised(x.double().cpu().numpy())[0]).cuda()
        args = (buf, None)
    else:
        c, s = random_mx(T, K, seed + 1)
        xv, args = values(c, s), (c, tiled(s))
    b = t.randn(N, generator=g, device="cuda") if bias else None
    y = t.full((T, max(ys, N)), 5.0, dtype=t.bfloat16, device="cuda")
    r = None
    if residual:
        r = t.randn(T, max(rs, N), generator=g, device="cuda", dtype=t.bfloat16)
        if alias:
            y[:, :N] = r[:, :N]
    shape = moe.mx_shape(T, N, K, kind, xs, ys, ys if alias else rs)
    ws = workspace(shape)
    wv = values(wc, wsc)
    ref = xv @ wv.T
    if bias:
        ref = ref + b.double()
    if residual:
        ref = ref + r[:, :N].double()
    moe.moe_mx_linear(shape, *args, wc, tiled(wsc), b, y if alias else r, y, ws)
    moe.moe_check_device_status(ws)
    err = (y[:, :N].double() - ref).abs()
    lim = bound(xv, wv, ref, b, None if r is None else r[:, :N])
    worst = (err / lim).max().item()
    assert worst <= 1, worst
    assert (y[:, N:] == 5).all()
    return y


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 32, 33, 64, 65, 127, 128, 129, 255, 256, 257, 300, 513])
def test_tokens(T, kind):
    product(T, 256, 512, kind)


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("N", [1, 2, 7, 127, 128, 129, 131, 1000])
def test_features(N, kind):
    for T in (3, 70, 140, 400):
        product(T, N, 256, kind, bias=True, residual=True)


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("K", [32, 64, 96, 128, 160, 192, 256, 288, 320, 480, 2048, 2080, 7168, 16384])
def test_widths(K, kind):
    for T in (5, 40, 200, 520):
        product(T, 200, K, kind, seed=K)


def test_strides():
    for T in (4, 24, 150, 300):
        product(T, 130, 256, xs=264, ys=137, rs=135, bias=True, residual=True)
        product(T, 128, 256, xs=512, ys=256, rs=140, residual=True)
        product(T, 130, 256, ys=130, residual=True, alias=True)
        product(T, 130, 256, "mxfp4", ys=132, residual=True, alias=True, rs=132)


def test_full_sizes():
    product(1, 9216, 7168)
    product(24, 7168, 7168, residual=True)
    product(256, 9216, 7168, "mxfp4")
    product(1003, 4099, 2080, bias=True)
    product(2500, 2304, 1792, bias=True, residual=True)
    product(777, 1021, 640, bias=True, residual=True)
    product(777, 1021, 640, rs=1022, ys=1024, residual=True)
    product(777, 1022, 640, rs=1023, ys=1029, residual=True)
    product(777, 1022, 640, ys=1027, residual=True, alias=True)
    product(4096, 1024, 7168)
    product(162, 128, 16352, "mxfp4")
    product(295, 135, 14912, bias=True, residual=True)
    product(700, 300, 8192)


@pytest.mark.parametrize("T", [1, 30, 100, 600])
def test_exact_integers(T):
    """Sums of small integers are exact in fp32 whatever their order: a misplaced row, code or scale shows as a
    whole number."""
    t = torch()
    K, N = 1056, 385
    g = t.Generator().manual_seed(T)
    x = t.randint(-2, 3, (T, K), generator=g).to(t.bfloat16).cuda()
    w = t.randint(-2, 3, (N, K), generator=g).to(t.bfloat16).cuda()
    wc, wsc = quantise(w, tiles=True)
    shape = moe.mx_shape(T, N, K)
    y = t.empty(T, N, dtype=t.bfloat16, device="cuda")
    ws = workspace(shape)
    moe.moe_mx_linear(shape, x, None, wc, wsc, None, None, y, ws)
    xv = quantised(x.double().cpu().numpy())[0]
    wv = quantised(w.double().cpu().numpy())[0]
    ref = t.from_numpy(xv @ wv.T).to(t.bfloat16)
    assert (y.cpu() == ref).all()


def test_one_element_at_a_time():
    """x with a single element finds each column of w, w's scales in every place of a tile."""
    t = torch()
    K, N = 320, 160
    wc, wsc = random_mx(N, K, 3, lo=100, hi=150)
    wt, wv = tiled(wsc), values(wc, wsc)
    for T in (16, 320):
        x = t.zeros(T, K, dtype=t.bfloat16, device="cuda")
        at = (t.arange(T, device="cuda") * 37 + 5) % K
        x[t.arange(T, device="cuda"), at] = 1
        shape = moe.mx_shape(T, N, K)
        y = t.empty(T, N, dtype=t.bfloat16, device="cuda")
        moe.moe_mx_linear(shape, x, None, wc, wt, None, None, y, workspace(shape))
        assert (y.double() == wv[:, at].T).all()


def test_nan_blocks_stay_in_their_rows():
    t = torch()
    for T in (3, 40, 200):
        x = t.randn(T, 256, device="cuda", dtype=t.bfloat16, generator=t.Generator(device="cuda").manual_seed(1))
        x[1, 70] = float("nan")
        x[2, 9] = float("inf")
        wc, wsc = random_mx(96, 256, 5)
        wsc[7, 3] = 255
        shape = moe.mx_shape(T, 96, 256)
        y = t.empty(T, 96, dtype=t.bfloat16, device="cuda")
        moe.moe_mx_linear(shape, x, None, wc, tiled(wsc), None, None, y, workspace(shape))
        bad = t.isnan(y)
        assert bad[1].all() and bad[2].all() and bad[:, 7].all()
        bad[1:3], bad[:, 7] = False, False
        assert not bad.any()


def test_repeats_bit_for_bit_and_in_graphs():
    t = torch()
    for T, N, K in ((1, 512, 4096), (24, 640, 2048), (200, 384, 1024), (700, 512, 768)):
        a = product(T, N, K, seed=9)
        b = product(T, N, K, seed=9)
        assert (a == b).all()
        wc, wsc = random_mx(N, K, 9)
        wt = tiled(wsc)
        shape = moe.mx_shape(T, N, K)
        ws = workspace(shape)
        x = t.zeros(T, K, dtype=t.bfloat16, device="cuda")
        y = t.empty(T, N, dtype=t.bfloat16, device="cuda")
        z = t.empty_like(y)
        moe.moe_mx_linear(shape, x, None, wc, wt, None, None, y, ws)
        t.cuda.synchronize()
        graph = t.cuda.CUDAGraph()
        with t.cuda.graph(graph):  # two calls in a row share the workspace
            moe.moe_mx_linear(shape, x, None, wc, wt, None, None, y, ws)
            moe.moe_mx_linear(shape, x, None, wc, wt, None, y, z, ws)
        x.copy_(t.randn(T, K, generator=t.Generator(device="cuda").manual_seed(9), device="cuda"))
        graph.replay()
        graph.replay()
        t.cuda.synchronize()
        moe.moe_check_device_status(ws)
        xv = t.from_numpy(quantised(x.double().cpu().numpy())[0]).cuda()
        ref = xv @ values(wc, wsc).T
        assert ((y.double() - ref).abs() <= bound(xv, values(wc, wsc), ref, None, None)).all()
        ref2 = ref + y.double()
        assert ((z.double() - ref2).abs() <= bound(xv, values(wc, wsc), ref2, None, y)).all()


@pytest.mark.parametrize("T", [1, 8, 40, 128, 300])
def test_weights_written_just_before(T):
    """A product right behind the kernel that quantises its weights reads the new ones, and one behind the
    kernel that writes its x."""
    t = torch()
    K, N = 2048, 4096
    codes = t.zeros(N, K // 2, dtype=t.uint8, device="cuda")
    r = moe.mx_rows(N, K, tiles=True)
    scales = t.zeros(moe.moe_mx_scale_bytes(r), dtype=t.uint8, device="cuda")
    x = t.ones(T, K, dtype=t.bfloat16, device="cuda")
    xc = t.zeros(T, K // 2, dtype=t.uint8, device="cuda")
    rx = moe.mx_rows(T, K, tiles=True)
    xs = t.zeros(moe.moe_mx_scale_bytes(rx), dtype=t.uint8, device="cuda")
    shape, quantised_shape = moe.mx_shape(T, N, K), moe.mx_shape(T, N, K, "mxfp4")
    ws, y = workspace(shape), t.empty(T, N, dtype=t.bfloat16, device="cuda")
    z = t.empty_like(y)
    weights = [t.full((N, K), v, dtype=t.bfloat16, device="cuda") for v in (1.0, 2.0, -0.5)]
    for w, v in zip(weights * 3, (1.0, 2.0, -0.5) * 3):
        moe.moe_mx_quantize(r, w, codes, scales)
        moe.moe_mx_linear(shape, x, None, codes, scales, None, None, y, ws)
        moe.moe_mx_quantize(rx, w[:T], xc, xs)
        moe.moe_mx_linear(quantised_shape, xc, xs, codes, scales, None, None, z, ws)
        assert (y == K * v).all() and (z == K * v * v).all()


def test_host_threads():
    """Calls of several host threads, with shapes that take different amounts of shared memory."""
    import threading
    t = torch()
    cases = [(1, 300, 4096), (2, 512, 1024), (1, 4096, 6144), (30, 256, 512), (200, 256, 512)]
    jobs, errors = [], []
    for i, (T, N, K) in enumerate(cases):
        wc, wsc = random_mx(N, K, i)
        x = t.randn(T, K, device="cuda", dtype=t.bfloat16)
        shape = moe.mx_shape(T, N, K)
        jobs.append((shape, x, wc, wsc, tiled(wsc), t.empty(T, N, dtype=t.bfloat16, device="cuda"),
                     workspace(shape), t.cuda.Stream()))
    t.cuda.synchronize()

    def work(job):
        shape, x, wc, _, wt, y, ws, st = job
        try:
            for _ in range(200):
                moe.moe_mx_linear(shape, x, None, wc, wt, None, None, y, ws, stream=st)
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    t.cuda.synchronize()
    assert not errors, errors
    for _, x, wc, wsc, _, y, ws, _ in jobs:
        moe.moe_check_device_status(ws)
        xv = t.from_numpy(quantised(x.double().cpu().numpy())[0]).cuda()
        wv = values(wc, wsc)
        ref = xv @ wv.T
        assert ((y.double() - ref).abs() <= bound(xv, wv, ref, None, None)).all()


def test_two_streams():
    t = torch()
    K, N = 1024, 512
    wc, wsc = random_mx(N, K, 11)
    wt, wv = tiled(wsc), values(wc, wsc)
    jobs = []
    t.cuda.synchronize()
    for i, T in enumerate((3, 20, 130, 40)):
        st = t.cuda.Stream()
        with t.cuda.stream(st):
            x = t.randn(T, K, device="cuda", dtype=t.bfloat16)
            shape = moe.mx_shape(T, N, K)
            y, ws = t.empty(T, N, dtype=t.bfloat16, device="cuda"), workspace(shape)
            for _ in range(5):
                moe.moe_mx_linear(shape, x, None, wc, wt, None, None, y, ws)
        jobs.append((x, y, ws))
    t.cuda.synchronize()
    for x, y, ws in jobs:
        moe.moe_check_device_status(ws)
        xv = t.from_numpy(quantised(x.double().cpu().numpy())[0]).cuda()
        ref = xv @ wv.T
        assert ((y.double() - ref).abs() <= bound(xv, wv, ref, None, None)).all()
