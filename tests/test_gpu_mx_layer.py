"""The MXFP4 projections and scored routing as layers use them: MxLinear, MoeLayer with a gate, weights quantised
here, and all of a decoder layer in a row (projection, attention, projection with the residual, gated MoE)."""
import numpy as np
import pytest

import oracle
import routed_expert_ffn_moe_gb300 as moe
import synth
from gpu_helpers import bf16_dev, bf16_host, torch
from mx_helpers import quantised, random_mx, selected, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from routed_expert_ffn_moe_gb300 import build
    build.build()
    moe.load()


def relative(a, b):
    return ((a.double() - b.double()).norm() / b.double().norm()).item()


def test_linear_layer():
    t = torch()
    g = t.Generator(device="cuda").manual_seed(1)
    w = t.randn(384, 512, generator=g, device="cuda").to(t.bfloat16)
    b = t.randn(384, generator=g, device="cuda")
    layer = moe.MxLinear.from_weight(w, b, max_tokens=300)
    wv = t.from_numpy(quantised(w.double().cpu().numpy())[0]).cuda()
    for T in (1, 20, 100, 300):
        x = t.randn(T, 640, generator=g, device="cuda").to(t.bfloat16)[:, :512]  # rows apart
        r = t.randn(T, 384, generator=g, device="cuda").to(t.bfloat16)
        out = t.empty(T, 400, dtype=t.bfloat16, device="cuda")[:, :384]
        y = layer.forward(x, r, out)
        assert y is out
        ref = t.from_numpy(quantised(x.double().cpu().numpy())[0]).cuda() @ wv.T + b.double() + r.double()
        assert relative(y, ref) < 2.0 ** -8  # one rounding to bf16, and fp32 sums
        y = layer.forward(x)
        assert y.data_ptr() == layer.y.data_ptr() and y.shape == (T, 384)
        assert relative(y, ref - r.double()) < 2.0 ** -8
    assert layer.forward(w[:0]).shape == (0, 384)
    layer.check()
    # from codes and scales in rows, and from fp32
    codes, scales = random_mx(384, 512, 4)
    y = moe.MxLinear(codes, scales).forward(w[:9])
    ref = t.from_numpy(quantised(w[:9].double().cpu().numpy())[0]).cuda() @ values(codes, scales).T
    assert relative(y, ref) < 2.0 ** -8
    assert (moe.MxLinear.from_weight(w.float()).forward(w[:9]) == moe.MxLinear.from_weight(w).forward(w[:9])).all()


def test_linear_layer_refuses():
    t = torch()
    codes, scales = random_mx(64, 128, 5)
    layer = moe.MxLinear(codes, scales, max_tokens=8)
    x = t.zeros(4, 128, dtype=t.bfloat16, device="cuda")
    for bad in (x.float(), x.cpu(), x[:, :64], x.t(), t.zeros(9, 128, dtype=t.bfloat16, device="cuda"), x[0],
                t.zeros(4, 256, dtype=t.bfloat16, device="cuda")[:, ::2]):
        with pytest.raises(ValueError):
            layer.forward(bad)
    with pytest.raises(ValueError):
        layer.forward(x, residual=t.zeros(3, 64, dtype=t.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        layer.forward(x, out=t.zeros(4, 64, device="cuda"))
    with pytest.raises(moe.MoeError):  # rows that do not start at 16 bytes
        layer.forward(t.zeros(4, 132, dtype=t.bfloat16, device="cuda")[:, :128])
    for kw in (dict(codes=codes.cpu()), dict(scales=scales[:, :2]), dict(codes=codes.short()),
               dict(bias=t.zeros(63, device="cuda")), dict(bias=t.zeros(64, device="cuda").double())):
        with pytest.raises(ValueError):
            moe.MxLinear(**{**dict(codes=codes, scales=scales), **kw})
    with pytest.raises(ValueError):
        moe.MxLinear.from_weight(t.zeros(64, 128, dtype=t.float16, device="cuda"))
    with pytest.raises(moe.MoeError):
        moe.MxLinear(t.zeros(64, 20, dtype=t.uint8, device="cuda"), t.zeros(64, 1, dtype=t.uint8, device="cuda"))


def gated_reference(cfg, inp, gate, sel):
    """The layer by its definition: fp64 scores, selection and the oracle's expert outputs."""
    x = oracle.bf16_to_f64(inp.x) if hasattr(oracle, "bf16_to_f64") else (
        inp.x.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    wg = (inp.wg.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    return selected(x @ wg.T, sel, cfg.k, **gate)


@pytest.mark.parametrize("wdtype", ["bf16", "mxfp4"])
def test_moe_layer_with_a_gate(wdtype):
    """Routing by the gate, then the same permutation, experts and combination as without one: the outputs are
    those of the separate calls on the gate's own choice."""
    t = torch()
    cfg = synth.get_config("tiny", wdtype=wdtype)
    inp = synth.host_inputs(cfg)
    raw = lambda a: t.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    w13, w2 = (np.stack([getattr(e, n) for e in inp.experts]) for n in ("w13", "w2"))
    if wdtype == "bf16":
        w = {"w13": bf16_dev(w13), "w2": bf16_dev(w2), "s13": None, "s2": None}
    else:
        w = {"w13": raw(w13), "w2": raw(w2), "s13": raw(np.stack([e.s13 for e in inp.experts])),
             "s2": raw(np.stack([e.s2 for e in inp.experts]))}
    sel = (np.random.default_rng(3).standard_normal(cfg.E) * 0.1).astype(np.float32)
    w.update(wg=bf16_dev(inp.wg), bias=None, sel_bias=raw(sel))
    kw = dict(score="sigmoid", n_group=4, topk_group=2, group_top=2, renorm=True, scale=2.5)
    gate = moe.gate_of(**kw)
    layer = moe.MoeLayer(cfg.T, cfg.d, cfg.E, cfg.k, cfg.f, cfg.n_shared, cfg.wdtype, w, gate=gate)
    x = bf16_dev(inp.x)
    y = layer.forward(x).clone()
    moe.moe_check_device_status(layer.ws)
    idx, wts = gated_reference(cfg, inp, kw, sel)
    np.testing.assert_array_equal(layer.topk_idx.cpu().numpy(), idx)
    assert np.abs(layer.topk_w.cpu().numpy() - wts).max() < 1e-5 * 2.5
    # the combination of the experts' outputs with these weights, in 64 bits
    yp = layer.y_perm.double()
    inv = layer.inv_slot.long().view(cfg.T, cfg.k)
    ref = yp[cfg.T * cfg.k:] + (layer.topk_w.double()[..., None] * yp[inv]).sum(1)
    assert ((y.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 1e-5 * ref.abs().max()).all()
    # the plain layer's choice differs, and a layer without a gate is what it was
    plain = moe.MoeLayer(cfg.T, cfg.d, cfg.E, cfg.k, cfg.f, cfg.n_shared, cfg.wdtype, w)
    yp = plain.forward(x)
    ref = oracle.moe_layer(cfg, inp)
    assert np.array_equal(plain.topk_idx.cpu().numpy(), ref["topk_idx"])
    assert relative(yp, t.from_numpy(ref["y"])[:].cuda()) < 1e-2
    assert bf16_host(y).shape == (cfg.T, cfg.d)


def test_experts_quantised_here():
    """Weights that moe_mx_quantize made serve the MXFP4 experts as the generator's own do, bit for bit."""
    t = torch()
    cfg = synth.get_config("tiny", wdtype="mxfp4")
    inp = synth.host_inputs(cfg)
    raw = lambda a: t.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    base = {"wg": bf16_dev(inp.wg), "bias": None}
    made = {k: raw(np.stack([getattr(e, k) for e in inp.experts])) for k in ("w13", "w2", "s13", "s2")}
    here = {}
    for name, rows, K, host in (("13", 2 * cfg.f, cfg.d, synth.host_w13_expert),
                                ("2", cfg.d, cfg.f, synth.host_w2_expert)):
        w = bf16_dev(np.stack([host(cfg, e) for e in range(cfg.E + 1)]))
        n = (cfg.E + 1) * rows
        codes = t.empty(cfg.E + 1, rows, K // 2, dtype=t.uint8, device="cuda")
        scales = t.empty(cfg.E + 1, rows, K // 32, dtype=t.uint8, device="cuda")
        moe.moe_mx_quantize(moe.mx_rows(n, K), w, codes, scales)
        here["w" + name], here["s" + name] = codes, scales
    x = bf16_dev(inp.x)
    ys = []
    for w in (made, here):
        layer = moe.MoeLayer(cfg.T, cfg.d, cfg.E, cfg.k, cfg.f, 1, "mxfp4", {**base, **w})
        ys.append(layer.forward(x).clone())
        moe.moe_check_device_status(layer.ws)
    assert (ys[0] == ys[1]).all()


@pytest.mark.parametrize("captured", [False, True])
def test_a_decoder_layer_in_a_row(captured):
    """Projection, attention, projection with the residual, gated MoE on one stream, with no wait between, against
    the same steps in 64 bits on what each step was given; prompts, then single tokens; also replayed."""
    t = torch()
    g = t.Generator(device="cuda").manual_seed(7)
    d, Hq, Hkv, D, E, k, f = 512, 8, 2, 64, 8, 2, 256
    bf = lambda *s: (t.randn(*s, generator=g, device="cuda") * 0.05).to(t.bfloat16)  # noqa: E731
    wq, wo = bf((Hq + 2 * Hkv) * D, d), bf(d, Hq * D)
    qkv_p, out_p = moe.MxLinear.from_weight(wq, max_tokens=256), moe.MxLinear.from_weight(wo, max_tokens=256)
    attn = moe.AttnLayer(Hq, Hkv, D, num_pages=40, max_pages=10, max_batch=2, max_tokens=256)
    weights = {"wg": bf(E, d), "bias": None, "w13": bf(E + 1, 2 * f, d), "w2": bf(E + 1, d, f), "s13": None,
               "s2": None, "sel_bias": t.randn(E, generator=g, device="cuda") * 0.05}
    table = t.randperm(40, generator=t.Generator().manual_seed(1))[:20].view(2, 10).to(t.int32).cuda()
    ints = lambda *v: t.tensor(v, dtype=t.int32, device="cuda")  # noqa: E731
    value = lambda m: t.from_numpy(quantised(m.double().cpu().numpy())[0]).cuda()  # noqa: E731
    wqv, wov = value(wq), value(wo)
    gate = moe.gate_of(n_group=4, topk_group=2, scale=2.5)
    lens = [0, 0]
    for new in ((90, 57), (1, 1), (1, 1)):
        T = sum(new)
        lens = [a + b for a, b in zip(lens, new)]
        x = bf(T, d) * 20
        layer = moe.MoeLayer(T, d, E, k, f, 1, "bf16", weights, gate=gate)
        kv_len = ints(*lens)
        q_start = ints(0, new[0], T) if T > 2 else None
        h = t.empty(T, d, dtype=t.bfloat16, device="cuda")

        def step():
            qkv = qkv_p.forward(x)
            o = attn.forward(qkv, table, kv_len, q_start)
            out_p.forward(o, x, h)
            return qkv, o, layer.forward(h)

        if captured:
            t.cuda.synchronize()
            graph = t.cuda.CUDAGraph()
            with t.cuda.graph(graph):
                qkv, o, y = step()
            graph.replay()
            graph.replay()  # the same places are written again
        else:
            qkv, o, y = step()
        t.cuda.synchronize()
        for layer_ in (qkv_p, out_p, attn):
            layer_.check()
        moe.moe_check_device_status(layer.ws)
        assert relative(qkv, value(x) @ wqv.T) < 2.0 ** -8
        assert relative(h, value(o) @ wov.T + x.double()) < 2.0 ** -8
        logits = h.double() @ weights["wg"].double().T
        idx, _ = selected(logits.cpu().numpy(), weights["sel_bias"].cpu().numpy(), k, n_group=4, topk_group=2)
        assert (layer.topk_idx.cpu().numpy() == idx).all(1).mean() > 0.98  # fp32 logits next to each other
        yp = layer.y_perm.double()
        ref = yp[T * k:] + (layer.topk_w.double()[..., None] * yp[layer.inv_slot.long().view(T, k)]).sum(1)
        assert relative(y, ref) < 2.0 ** -8


def test_the_example_runs_in_4_bits():
    import importlib.util
    import os
    at = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decoder_block.py")
    spec = importlib.util.spec_from_file_location("decoder_block", at)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    torch().manual_seed(0)
    # steps and whole prompts round to bf16 at the same places, but a value that falls on the other side of an
    # E2M1 border moves by a quarter: the two agree only roughly
    assert np.isfinite(example.run(fp4=True, kv_dtype="fp8"))
