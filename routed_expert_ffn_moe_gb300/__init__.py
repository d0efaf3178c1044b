"""Python binding of the GB300 routed-expert MoE FFN library (include/moe.h).

Argument marshalling only: every step of the layer runs in the CUDA kernels of
libmoe_gb300.so. Tensors are torch CUDA tensors (PyTorch provides device memory and streams);
the functions below pass their device pointers to the C ABI. There is no CPU fallback: if the
library is missing or was not built, every call raises.
"""
from __future__ import annotations

import ctypes
import os

__all__ = ["MoeError", "MoeShape", "MOE_W_BF16", "MOE_W_FP8_E4M3_B128", "MOE_W_MXFP4_E8M0_B32",
           "load", "lib_path",
           "moe_workspace_size", "moe_route", "moe_route_hash", "moe_route_noalloc", "moe_permute",
           "moe_expert_ffn", "moe_combine", "moe_forward",
           "moe_check_device_status", "moe_selftest_bounded_wait", "moe_profile_enable",
           "moe_profile_read",
           "moe_last_error_string", "shape_of", "MoeLayer", "EXPORTED",
           "MoeAttnShape", "MOE_KV_BF16", "MOE_KV_FP8_E4M3", "attn_shape",
           "moe_attn_workspace_size", "moe_attn_workspace_zero_bytes", "moe_attn_append",
           "moe_attn_decode", "moe_attn_prefill", "AttnLayer",
           "MoeGate", "MOE_SCORE_SOFTMAX", "MOE_SCORE_SIGMOID", "gate_of", "moe_route_select",
           "moe_route_gate", "MoeMxRows", "MoeMxShape", "MOE_T_BF16", "MOE_T_F32", "MOE_T_MXFP4",
           "mx_rows", "mx_shape", "moe_mx_scale_bytes", "moe_mx_quantize", "moe_mx_dequantize",
           "moe_mx_tile_scales", "moe_mx_linear_workspace_size", "moe_mx_linear", "MxLinear"]

MOE_W_BF16, MOE_W_FP8_E4M3_B128, MOE_W_MXFP4_E8M0_B32 = 0, 1, 2
WDTYPES = {"bf16": MOE_W_BF16, "fp8": MOE_W_FP8_E4M3_B128, "mxfp4": MOE_W_MXFP4_E8M0_B32}
MOE_KV_BF16, MOE_KV_FP8_E4M3 = 0, 1
KV_DTYPES = {"bf16": MOE_KV_BF16, "fp8": MOE_KV_FP8_E4M3}
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
SCORES = {"softmax": MOE_SCORE_SOFTMAX, "sigmoid": MOE_SCORE_SIGMOID}
MOE_T_BF16, MOE_T_F32, MOE_T_MXFP4 = 0, 1, 2
MX_DTYPES = {"bf16": MOE_T_BF16, "f32": MOE_T_F32, "mxfp4": MOE_T_MXFP4}
STATUS = {0: "MOE_OK", -1: "MOE_ERR_INVALID_ARG", -2: "MOE_ERR_UNSUPPORTED",
          -3: "MOE_ERR_WORKSPACE", -4: "MOE_ERR_CUDA", -5: "MOE_ERR_DEVICE_TIMEOUT",
          -6: "MOE_ERR_DEVICE_BOUNDS"}
EXPORTED = ("moe_workspace_size", "moe_route", "moe_route_hash", "moe_route_noalloc", "moe_permute",
            "moe_expert_ffn",
            "moe_combine", "moe_forward",
            "moe_check_device_status", "moe_selftest_bounded_wait", "moe_profile_enable",
            "moe_profile_read", "moe_last_error_string",
            "moe_attn_workspace_size", "moe_attn_workspace_zero_bytes", "moe_attn_append",
            "moe_attn_decode", "moe_attn_prefill",
            "moe_route_select", "moe_route_gate", "moe_mx_scale_bytes", "moe_mx_quantize",
            "moe_mx_dequantize", "moe_mx_tile_scales", "moe_mx_linear_workspace_size",
            "moe_mx_linear")

_PKG = os.path.dirname(os.path.abspath(__file__))


def lib_path() -> str:
    return os.path.join(_PKG, "libmoe_gb300.so")


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str, msg: str):
        super().__init__(f"{where}: {STATUS.get(status, status)}: {msg}")
        self.status = status


class MoeShape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("E", ctypes.c_int32),
                ("k", ctypes.c_int32), ("f", ctypes.c_int32), ("n_shared", ctypes.c_int32),
                ("wdtype", ctypes.c_int32)]


class MoeAttnShape(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in
                 ("T", "B", "Hq", "Hkv", "D", "kv_dtype", "page_size", "max_pages", "num_pages",
                  "window", "n_sink", "rot_dim", "rot_pairs", "max_pos")]
                + [("scale", ctypes.c_float), ("eps", ctypes.c_float)]
                + [(n, ctypes.c_int64) for n in
                   ("q_stride", "k_stride", "v_stride", "qr_stride", "o_stride", "page_stride",
                    "head_stride", "token_stride")])


class MoeGate(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("score", "n_group", "topk_group", "group_top", "renorm")]
                + [("scale", ctypes.c_float)])


class MoeMxRows(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("rows", "K", "dtype", "tiles")]
                + [("stride", ctypes.c_int64)])


class MoeMxShape(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("T", "N", "K", "x_dtype")]
                + [(n, ctypes.c_int64) for n in ("x_stride", "y_stride", "r_stride")])


_lib = None


def load():
    """Loads libmoe_gb300.so. Raises if it has not been built (no fallback exists)."""
    global _lib
    if _lib is not None:
        return _lib
    path = lib_path()
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it first "
                          "(python -m routed_expert_ffn_moe_gb300.build or __graft_entry__.build())")
    L = ctypes.CDLL(path)
    vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    shp = ctypes.POINTER(MoeShape)
    L.moe_workspace_size.restype = sz
    L.moe_workspace_size.argtypes = [shp]
    L.moe_route.restype = i32
    L.moe_route.argtypes = [shp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.moe_route_hash.restype = i32
    L.moe_route_hash.argtypes = [shp, vp, vp, vp, vp, vp, ctypes.c_int32, vp, vp, vp, sz, vp]
    L.moe_route_noalloc.restype = i32
    L.moe_route_noalloc.argtypes = [shp, vp, vp, vp, vp, vp, vp]
    L.moe_permute.restype = i32
    L.moe_permute.argtypes = [shp, vp, vp, vp, vp, vp, sz, vp]
    L.moe_expert_ffn.restype = i32
    L.moe_expert_ffn.argtypes = [shp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.moe_combine.restype = i32
    L.moe_combine.argtypes = [shp, vp, vp, vp, vp, vp, sz, vp]
    L.moe_forward.restype = i32
    L.moe_forward.argtypes = [shp] + [vp] * 15 + [sz, vp]
    L.moe_check_device_status.restype = i32
    L.moe_check_device_status.argtypes = [vp, vp]
    L.moe_selftest_bounded_wait.restype = i32
    L.moe_selftest_bounded_wait.argtypes = [vp, ctypes.c_uint32, vp]
    L.moe_profile_enable.restype = i32
    L.moe_profile_enable.argtypes = [i32]
    L.moe_profile_read.restype = i32
    L.moe_profile_read.argtypes = [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_double),
                                   ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_int64)]
    ashp = ctypes.POINTER(MoeAttnShape)
    L.moe_attn_workspace_size.restype = sz
    L.moe_attn_workspace_size.argtypes = [ashp, i32]
    L.moe_attn_workspace_zero_bytes.restype = sz
    L.moe_attn_workspace_zero_bytes.argtypes = []
    L.moe_attn_append.restype = i32
    L.moe_attn_append.argtypes = [ashp] + [vp] * 16 + [sz, vp]
    L.moe_attn_decode.restype = i32
    L.moe_attn_decode.argtypes = [ashp] + [vp] * 10 + [sz, vp]
    L.moe_attn_prefill.restype = i32
    L.moe_attn_prefill.argtypes = [ashp] + [vp] * 11 + [sz, vp]
    gate = ctypes.POINTER(MoeGate)
    L.moe_route_select.restype = i32
    L.moe_route_select.argtypes = [shp, gate] + [vp] * 5
    L.moe_route_gate.restype = i32
    L.moe_route_gate.argtypes = [shp, gate] + [vp] * 7 + [sz, vp]
    rows, mshp = ctypes.POINTER(MoeMxRows), ctypes.POINTER(MoeMxShape)
    L.moe_mx_scale_bytes.restype = sz
    L.moe_mx_scale_bytes.argtypes = [rows]
    L.moe_mx_quantize.restype = i32
    L.moe_mx_quantize.argtypes = [rows] + [vp] * 4
    L.moe_mx_dequantize.restype = i32
    L.moe_mx_dequantize.argtypes = [rows] + [vp] * 4
    L.moe_mx_tile_scales.restype = i32
    L.moe_mx_tile_scales.argtypes = [rows] + [vp] * 3
    L.moe_mx_linear_workspace_size.restype = sz
    L.moe_mx_linear_workspace_size.argtypes = [mshp]
    L.moe_mx_linear.restype = i32
    L.moe_mx_linear.argtypes = [mshp] + [vp] * 8 + [sz, vp]
    L.moe_last_error_string.restype = ctypes.c_char_p
    L.moe_last_error_string.argtypes = []
    _lib = L
    return L


def _ptr(t):
    """Device pointer of a torch tensor (or an int address, or None)."""
    if t is None:
        return None
    try:
        return t.data_ptr()
    except AttributeError:
        return t


def _current_stream():
    """The current torch stream's handle, without the Stream object where torch offers that."""
    global _current_stream
    import torch
    try:
        raw, dev = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
        raw(dev())
        _current_stream = lambda: raw(dev())                            # noqa: E731
    except AttributeError:
        _current_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
    return _current_stream()


def _stream(stream):
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int, where: str):
    if rc != 0:
        raise MoeError(rc, where, load().moe_last_error_string().decode(errors="replace"))


def shape_of(T, d, E, k, f, n_shared=1, wdtype=MOE_W_BF16) -> MoeShape:
    if isinstance(wdtype, str):
        wdtype = WDTYPES[wdtype]
    return MoeShape(T, d, E, k, f, n_shared, wdtype)


def moe_last_error_string() -> str:
    return load().moe_last_error_string().decode(errors="replace")


def moe_workspace_size(shape: MoeShape) -> int:
    return int(load().moe_workspace_size(ctypes.byref(shape)))


def _ws(ws):
    return _ptr(ws), getattr(ws, "nbytes", 0)


def moe_route(shape, x, wg, bias, topk_idx, topk_w, ws, stream=None, ws_bytes=None):
    wp, wb = _ws(ws)
    _check(load().moe_route(ctypes.byref(shape), _ptr(x), _ptr(wg), _ptr(bias), _ptr(topk_idx),
                            _ptr(topk_w), wp, wb if ws_bytes is None else ws_bytes,
                            _stream(stream)), "moe_route")


def moe_route_hash(shape, x, wg, bias, token_ids, tid2eid, topk_idx, topk_w, ws, stream=None,
                   ws_bytes=None):
    """Hash routing: experts from tid2eid [vocab, k] by token id, the soft router's gate."""
    wp, wb = _ws(ws)
    _check(load().moe_route_hash(ctypes.byref(shape), _ptr(x), _ptr(wg), _ptr(bias),
                                 _ptr(token_ids), _ptr(tid2eid), int(tid2eid.shape[0]),
                                 _ptr(topk_idx), _ptr(topk_w), wp,
                                 wb if ws_bytes is None else ws_bytes, _stream(stream)),
           "moe_route_hash")


def moe_route_noalloc(shape, x, wg, bias, topk_idx, topk_w, stream=None):
    """moe_route without a workspace (for callers that cannot allocate device memory): the
    library keeps the logits in a fixed 4 MiB device array, so T*E must be <= 2^20."""
    _check(load().moe_route_noalloc(ctypes.byref(shape), _ptr(x), _ptr(wg), _ptr(bias),
                                    _ptr(topk_idx), _ptr(topk_w), _stream(stream)),
           "moe_route_noalloc")


def moe_permute(shape, topk_idx, expert_offsets, perm_token, inv_slot, ws, stream=None,
                ws_bytes=None):
    wp, wb = _ws(ws)
    _check(load().moe_permute(ctypes.byref(shape), _ptr(topk_idx), _ptr(expert_offsets),
                              _ptr(perm_token), _ptr(inv_slot), wp,
                              wb if ws_bytes is None else ws_bytes, _stream(stream)), "moe_permute")


def moe_expert_ffn(shape, x, perm_token, expert_offsets, w13, s13, w2, s2, y_perm, ws,
                   stream=None, ws_bytes=None):
    wp, wb = _ws(ws)
    _check(load().moe_expert_ffn(ctypes.byref(shape), _ptr(x), _ptr(perm_token),
                                 _ptr(expert_offsets), _ptr(w13), _ptr(s13), _ptr(w2), _ptr(s2),
                                 _ptr(y_perm), wp, wb if ws_bytes is None else ws_bytes,
                                 _stream(stream)), "moe_expert_ffn")


def moe_combine(shape, y_perm, inv_slot, topk_w, y, ws, stream=None, ws_bytes=None):
    wp, wb = _ws(ws)
    _check(load().moe_combine(ctypes.byref(shape), _ptr(y_perm), _ptr(inv_slot), _ptr(topk_w),
                              _ptr(y), wp, wb if ws_bytes is None else ws_bytes, _stream(stream)),
           "moe_combine")


def moe_forward(shape, x, wg, bias, w13, s13, w2, s2, topk_idx, topk_w, expert_offsets,
                perm_token, inv_slot, y_perm, y, ws, stream=None, ws_bytes=None):
    """The four calls in one, with the shared expert's FFN overlapped with the routing."""
    wp, wb = _ws(ws)
    _check(load().moe_forward(ctypes.byref(shape), _ptr(x), _ptr(wg), _ptr(bias), _ptr(w13),
                              _ptr(s13), _ptr(w2), _ptr(s2), _ptr(topk_idx), _ptr(topk_w),
                              _ptr(expert_offsets), _ptr(perm_token), _ptr(inv_slot),
                              _ptr(y_perm), _ptr(y), wp, wb if ws_bytes is None else ws_bytes,
                              _stream(stream)), "moe_forward")


def moe_check_device_status(ws, stream=None):
    _check(load().moe_check_device_status(_ptr(ws), _stream(stream)), "moe_check_device_status")


def moe_selftest_bounded_wait(ws, limit_us, stream=None):
    """Launches a kernel whose wait never completes; after `limit_us` it records
    MOE_ERR_DEVICE_TIMEOUT in ws's status word (read it with moe_check_device_status)."""
    _check(load().moe_selftest_bounded_wait(_ptr(ws), int(limit_us), _stream(stream)),
           "moe_selftest_bounded_wait")


def moe_profile_enable(on: bool = True):
    _check(load().moe_profile_enable(1 if on else 0), "moe_profile_enable")


def moe_profile_read() -> dict:
    up, dn = ctypes.c_double(), ctypes.c_double()
    calls, launches = ctypes.c_int64(), ctypes.c_int64()
    _check(load().moe_profile_read(ctypes.byref(up), ctypes.byref(dn), ctypes.byref(calls),
                                   ctypes.byref(launches)), "moe_profile_read")
    return {"ms_gate_up": up.value, "ms_down": dn.value, "ffn_calls": calls.value,
            "kernel_launches": launches.value}


def attn_shape(T, B, Hq, Hkv, D, kv_dtype="bf16", page_size=16, max_pages=1, num_pages=1,
               window=0, n_sink=0, rot_dim=0, rot_pairs=False, max_pos=0, scale=0.0, eps=1e-6,
               q_stride=0, k_stride=0, v_stride=0, qr_stride=0, o_stride=0, page_stride=0,
               head_stride=0, token_stride=0) -> MoeAttnShape:
    """moe_attn_shape; a scale or stride of 0 is the default (1/sqrt(D), packed)."""
    if isinstance(kv_dtype, str):
        kv_dtype = KV_DTYPES[kv_dtype]
    return MoeAttnShape(T, B, Hq, Hkv, D, kv_dtype, page_size, max_pages, num_pages, window,
                        n_sink, rot_dim, int(rot_pairs), max_pos, scale, eps, q_stride, k_stride,
                        v_stride, qr_stride, o_stride, page_stride, head_stride, token_stride)


def moe_attn_workspace_size(shape: MoeAttnShape, prefill: bool = False) -> int:
    return int(load().moe_attn_workspace_size(ctypes.byref(shape), int(prefill)))


def moe_attn_workspace_zero_bytes() -> int:
    return int(load().moe_attn_workspace_zero_bytes())


def moe_attn_append(shape, q, k, v, q_norm, k_norm, cos_sin, positions, block_table, kv_len,
                    q_start, k_scale, v_scale, q_out, k_cache, v_cache, ws, stream=None,
                    ws_bytes=None):
    """Per-head norms, rotation and append to the paged cache; q_out is the rotated q."""
    wp, wb = _ws(ws)
    _check(load().moe_attn_append(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(q_norm),
                                  _ptr(k_norm), _ptr(cos_sin), _ptr(positions),
                                  _ptr(block_table), _ptr(kv_len), _ptr(q_start), _ptr(k_scale),
                                  _ptr(v_scale), _ptr(q_out), _ptr(k_cache), _ptr(v_cache), wp,
                                  wb if ws_bytes is None else ws_bytes, _stream(stream)),
           "moe_attn_append")


def moe_attn_decode(shape, q, k_cache, v_cache, k_scale, v_scale, block_table, kv_len, o, lse, ws,
                    stream=None, ws_bytes=None):
    """Attention of one new token per sequence over the paged cache."""
    wp, wb = _ws(ws)
    _check(load().moe_attn_decode(ctypes.byref(shape), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                  _ptr(k_scale), _ptr(v_scale), _ptr(block_table), _ptr(kv_len),
                                  _ptr(o), _ptr(lse), wp, wb if ws_bytes is None else ws_bytes,
                                  _stream(stream)), "moe_attn_decode")


def moe_attn_prefill(shape, q, k_cache, v_cache, k_scale, v_scale, block_table, kv_len, q_start,
                     o, lse, ws, stream=None, ws_bytes=None):
    """Attention of a ragged step of new tokens over the paged cache (which holds them already)."""
    wp, wb = _ws(ws)
    _check(load().moe_attn_prefill(ctypes.byref(shape), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                   _ptr(k_scale), _ptr(v_scale), _ptr(block_table), _ptr(kv_len),
                                   _ptr(q_start), _ptr(o), _ptr(lse), wp,
                                   wb if ws_bytes is None else ws_bytes, _stream(stream)),
           "moe_attn_prefill")


def gate_of(score="sigmoid", n_group=1, topk_group=1, group_top=2, renorm=True,
            scale=1.0) -> MoeGate:
    """moe_gate; score is "softmax", "sigmoid" or a MOE_SCORE_ number."""
    return MoeGate(SCORES[score] if isinstance(score, str) else score, n_group, topk_group,
                   group_top, int(renorm), scale)


def moe_route_select(shape, gate, logits, sel_bias, topk_idx, topk_w, stream=None):
    """The scored selection of each token's k experts from its logits [T, E] fp32."""
    _check(load().moe_route_select(ctypes.byref(shape), ctypes.byref(gate), _ptr(logits),
                                   _ptr(sel_bias), _ptr(topk_idx), _ptr(topk_w), _stream(stream)),
           "moe_route_select")


def moe_route_gate(shape, gate, x, wg, bias, sel_bias, topk_idx, topk_w, ws, stream=None,
                   ws_bytes=None):
    """The router with scored selection: moe_route's logits, then moe_route_select."""
    wp, wb = _ws(ws)
    _check(load().moe_route_gate(ctypes.byref(shape), ctypes.byref(gate), _ptr(x), _ptr(wg),
                                 _ptr(bias), _ptr(sel_bias), _ptr(topk_idx), _ptr(topk_w), wp,
                                 wb if ws_bytes is None else ws_bytes, _stream(stream)),
           "moe_route_gate")


def mx_rows(rows, K, dtype="bf16", tiles=False, stride=0) -> MoeMxRows:
    """moe_mx_rows; a stride of 0 is K."""
    return MoeMxRows(rows, K, MX_DTYPES[dtype] if isinstance(dtype, str) else dtype, int(tiles),
                     stride)


def mx_shape(T, N, K, x_dtype="bf16", x_stride=0, y_stride=0, r_stride=0) -> MoeMxShape:
    """moe_mx_shape; a stride of 0 is the packed one."""
    return MoeMxShape(T, N, K, MX_DTYPES[x_dtype] if isinstance(x_dtype, str) else x_dtype,
                      x_stride, y_stride, r_stride)


def moe_mx_scale_bytes(rows: MoeMxRows) -> int:
    return int(load().moe_mx_scale_bytes(ctypes.byref(rows)))


def moe_mx_quantize(rows, x, codes, scales, stream=None):
    """x [rows, K] to MXFP4 codes [rows, K/2] and scales (moe_mx_scale_bytes)."""
    _check(load().moe_mx_quantize(ctypes.byref(rows), _ptr(x), _ptr(codes), _ptr(scales),
                                  _stream(stream)), "moe_mx_quantize")


def moe_mx_dequantize(rows, codes, scales, y, stream=None):
    """The values of MXFP4 rows into y [rows, K]."""
    _check(load().moe_mx_dequantize(ctypes.byref(rows), _ptr(codes), _ptr(scales), _ptr(y),
                                    _stream(stream)), "moe_mx_dequantize")


def moe_mx_tile_scales(rows, scales, tiles, stream=None):
    """Scales in rows to scales in tiles."""
    _check(load().moe_mx_tile_scales(ctypes.byref(rows), _ptr(scales), _ptr(tiles),
                                     _stream(stream)), "moe_mx_tile_scales")


def moe_mx_linear_workspace_size(shape: MoeMxShape) -> int:
    return int(load().moe_mx_linear_workspace_size(ctypes.byref(shape)))


def moe_mx_linear(shape, x, x_scales, w, w_scales, bias, residual, y, ws, stream=None,
                  ws_bytes=None):
    """y = x w^T + bias + residual with both matrices in MXFP4."""
    wp, wb = _ws(ws)
    _check(load().moe_mx_linear(ctypes.byref(shape), _ptr(x), _ptr(x_scales), _ptr(w),
                                _ptr(w_scales), _ptr(bias), _ptr(residual), _ptr(y), wp,
                                wb if ws_bytes is None else ws_bytes, _stream(stream)),
           "moe_mx_linear")


class MoeLayer:
    """The four calls chained on one stream with buffers allocated once (torch, on `device`).

    weights: dict with wg [E,d] bf16, bias [E] f32 or None, w13, w2 (bf16, uint8 E4M3 codes or
    uint8 MXFP4 code pairs), s13, s2 (fp32 block scales, uint8 E8M0 scales, or None). `forward(x)` returns y [T,d] bf16; intermediate tensors
    stay available as attributes (topk_idx, topk_w, expert_offsets, perm_token, inv_slot, y_perm).

    gate: a MoeGate (gate_of) for scored routing (moe_route_gate) instead of moe_route; the weights
    may then hold sel_bias [E] f32.
    """

    def __init__(self, T, d, E, k, f, n_shared, wdtype, weights, device="cuda", gate=None):
        import torch
        self.shape = shape_of(T, d, E, k, f, n_shared, wdtype)
        self.gate = gate
        self.w = weights
        dev = torch.device(device)
        slots = T * k + n_shared * T
        self.ws = torch.empty(max(moe_workspace_size(self.shape), 256), dtype=torch.uint8, device=dev)
        self.ws[:4].zero_()
        self.topk_idx = torch.empty(T, k, dtype=torch.int32, device=dev)
        self.topk_w = torch.empty(T, k, dtype=torch.float32, device=dev)
        self.expert_offsets = torch.empty(E + 2, dtype=torch.int32, device=dev)
        self.perm_token = torch.empty(max(T * k, 1), dtype=torch.int32, device=dev)
        self.inv_slot = torch.empty(max(T * k, 1), dtype=torch.int32, device=dev)
        self.y_perm = torch.empty(max(slots, 1), d, dtype=torch.float32, device=dev)
        self.y = torch.empty(T, d, dtype=torch.bfloat16, device=dev)

    def forward(self, x, stream=None):
        """The layer through moe_forward (one call; the shared expert overlaps the routing), or with a
        gate as the four calls."""
        w = self.w
        if self.gate is not None:
            return self.forward_steps(x, stream)
        moe_forward(self.shape, x, w["wg"], w.get("bias"), w["w13"], w.get("s13"), w["w2"],
                    w.get("s2"), self.topk_idx, self.topk_w, self.expert_offsets, self.perm_token,
                    self.inv_slot, self.y_perm, self.y, self.ws, stream)
        return self.y

    def forward_hash(self, x, token_ids, tid2eid, stream=None):
        """The layer with hash routing (moe_route_hash, then permute, expert FFN, combine)."""
        w, s = self.w, self.shape
        moe_route_hash(s, x, w["wg"], w.get("bias"), token_ids, tid2eid, self.topk_idx,
                       self.topk_w, self.ws, stream)
        moe_permute(s, self.topk_idx, self.expert_offsets, self.perm_token, self.inv_slot, self.ws,
                    stream)
        moe_expert_ffn(s, x, self.perm_token, self.expert_offsets, w["w13"], w.get("s13"),
                       w["w2"], w.get("s2"), self.y_perm, self.ws, stream)
        moe_combine(s, self.y_perm, self.inv_slot, self.topk_w, self.y, self.ws, stream)
        return self.y

    def forward_steps(self, x, stream=None):
        """The layer as the four separate calls."""
        w, s = self.w, self.shape
        if self.gate is not None:
            moe_route_gate(s, self.gate, x, w["wg"], w.get("bias"), w.get("sel_bias"),
                           self.topk_idx, self.topk_w, self.ws, stream)
        else:
            moe_route(s, x, w["wg"], w.get("bias"), self.topk_idx, self.topk_w, self.ws, stream)
        moe_permute(s, self.topk_idx, self.expert_offsets, self.perm_token, self.inv_slot, self.ws,
                    stream)
        moe_expert_ffn(s, x, self.perm_token, self.expert_offsets, w["w13"], w.get("s13"),
                       w["w2"], w.get("s2"), self.y_perm, self.ws, stream)
        moe_combine(s, self.y_perm, self.inv_slot, self.topk_w, self.y, self.ws, stream)
        return self.y


class AttnLayer:
    """The attention of one decoder layer between its qkv and its output projection, with the cache,
    the rotation table and the workspace allocated once (torch, on `device`).

    `forward(qkv, block_table, kv_len, q_start)` takes a step's projections, one row
    [(Hq + 2 Hkv) * D] bf16 a token (query heads, key heads, value heads), appends keys and values
    to the cache and returns o [T, Hq * D] bf16: attention of one token a sequence where q_start is
    None, else of the ragged step that q_start [B + 1] describes. kv_len [B] counts the step's
    tokens; block_table [B, max_pages] names each sequence's pages. All three are int32, packed, on the
    layer's device; the rows of qkv may lie apart. Tensors of another type or layout raise ValueError;
    out-of-range pages, lengths and positions are reported by `check()`. o is the layer's own buffer:
    the next forward overwrites it. Optional: positions [T] int32 (of the rotation), lse [T, Hq] fp32
    (written).

    max_batch and max_tokens bound the sequences and tokens of a step. norms: (q_norm, k_norm), [D]
    bf16 each, or None; scales: (k_scale, v_scale), [Hkv] fp32 each, for an "fp8" cache. For such a
    cache, and for pages that are no multiple of 16 tokens, the workspace also holds the bf16 keys and
    values of max_batch sequences of max_pages * page_size places, unpacked by steps with q_start.
    """

    def __init__(self, Hq, Hkv, D, num_pages, page_size=16, max_pages=256, max_batch=64,
                 max_tokens=4096, kv_dtype="bf16", window=0, n_sink=0, rot_dim=None,
                 rot_pairs=False, rope_base=10000.0, norms=None, scales=None, scale=0.0, eps=1e-6,
                 device="cuda"):
        import torch
        self.Hq, self.Hkv, self.D = Hq, Hkv, D
        row = (Hq + 2 * Hkv) * D
        self.max_batch, self.max_tokens, self.max_pages = max_batch, max_tokens, max_pages
        self.q_norm, self.k_norm = norms or (None, None)
        self.k_scale, self.v_scale = scales or (None, None)
        self._i32, self._bf16, self._f32 = torch.int32, torch.bfloat16, torch.float32
        rot_dim = D if rot_dim is None else rot_dim
        max_pos = page_size * max_pages
        self._kw = dict(Hq=Hq, Hkv=Hkv, D=D, kv_dtype=kv_dtype, page_size=page_size,
                        max_pages=max_pages, num_pages=num_pages, window=window, n_sink=n_sink,
                        rot_dim=rot_dim, rot_pairs=rot_pairs, max_pos=max_pos, scale=scale,
                        eps=eps)
        self._row = row
        dev = torch.device(device)
        dt = torch.bfloat16 if kv_dtype in ("bf16", MOE_KV_BF16) else torch.uint8
        self.k_cache = torch.zeros(num_pages, Hkv, page_size, D, dtype=dt, device=dev)
        self.v_cache = torch.zeros_like(self.k_cache)
        self._dev = self.k_cache.device
        for name, t, kind, n in (("q_norm", self.q_norm, self._bf16, D),
                                 ("k_norm", self.k_norm, self._bf16, D),
                                 ("k_scale", self.k_scale, self._f32, Hkv),
                                 ("v_scale", self.v_scale, self._f32, Hkv)):
            self._packed(name, t, kind, n)
        freq = rope_base ** (-torch.arange(rot_dim // 2, dtype=torch.float64) / max(rot_dim // 2, 1))
        ang = torch.arange(max_pos, dtype=torch.float64)[:, None] * freq
        self.cos_sin = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous().to(dev)
        n = moe_attn_workspace_size(attn_shape(T=max_tokens, B=max_batch, **self._kw), True)
        if n == 0:
            raise MoeError(-1, "AttnLayer", moe_last_error_string())
        self.ws = torch.empty(n, dtype=torch.uint8, device=dev)
        self.ws[:moe_attn_workspace_zero_bytes()].zero_()
        self.q_rot = torch.empty(max_tokens, Hq * D, dtype=torch.bfloat16, device=dev)
        self.o = torch.empty(max_tokens, Hq * D, dtype=torch.bfloat16, device=dev)
        self._shapes = {}

    def _packed(self, name, t, dtype, n):
        """Refuses a tensor whose first n elements do not lie in a row as `dtype` on the device."""
        if t is None or isinstance(t, int):  # an int is an address
            return
        if t.dtype != dtype or t.device != self._dev or t.numel() < n or not t.is_contiguous():
            raise ValueError(f"{name}: {t.dtype}, {tuple(t.shape)}, strides {t.stride()} on {t.device}: "
                             f"{n} packed elements of {dtype} on {self._dev} are needed")

    def _rows_apart(self, qkv, T):
        """The distance of qkv's rows, each (Hq + 2 Hkv) * D bf16 in a row."""
        row = self._row
        if qkv.dtype == self._bf16 and qkv.device == self._dev and qkv.numel() == T * row:
            if qkv.is_contiguous():
                return row
            if qkv[0].is_contiguous() and qkv.stride(0) >= row:
                return qkv.stride(0)
        raise ValueError(f"qkv: {qkv.dtype}, {tuple(qkv.shape)}, strides {qkv.stride()} on "
                         f"{qkv.device}: rows of {row} packed bf16 on {self._dev} are needed")

    def forward(self, qkv, block_table, kv_len, q_start=None, positions=None, lse=None, stream=None):
        T, B = qkv.shape[0], kv_len.shape[0]
        if T > self.max_tokens or B > self.max_batch or block_table.shape[1] != self.max_pages:
            raise ValueError(f"a step of {T} tokens, {B} sequences and tables of "
                             f"{block_table.shape[1]} pages: the layer was made for "
                             f"{self.max_tokens}, {self.max_batch} and {self.max_pages}")
        apart = self._rows_apart(qkv, T)
        self._packed("block_table", block_table, self._i32, B * self.max_pages)
        self._packed("kv_len", kv_len, self._i32, B)
        self._packed("q_start", q_start, self._i32, B + 1)
        self._packed("positions", positions, self._i32, T)
        self._packed("lse", lse, self._f32, T * self.Hq)
        s = self._shapes.get((T, B, apart))
        if s is None:
            if len(self._shapes) >= 1024:
                self._shapes.clear()
            s = self._shapes[(T, B, apart)] = attn_shape(T=T, B=B, q_stride=apart, k_stride=apart,
                                                         v_stride=apart, **self._kw)
        nq, nk = self.Hq * self.D, self.Hkv * self.D
        at = qkv.data_ptr()
        q, k, v = (at, at + 2 * nq, at + 2 * (nq + nk)) if T else (None, None, None)
        o = self.o[:T]
        moe_attn_append(s, q, k, v, self.q_norm, self.k_norm, self.cos_sin, positions, block_table,
                        kv_len, q_start, self.k_scale, self.v_scale, self.q_rot, self.k_cache,
                        self.v_cache, self.ws, stream)
        if q_start is None:
            moe_attn_decode(s, self.q_rot, self.k_cache, self.v_cache, self.k_scale, self.v_scale,
                            block_table, kv_len, o, lse, self.ws, stream)
        else:
            moe_attn_prefill(s, self.q_rot, self.k_cache, self.v_cache, self.k_scale, self.v_scale,
                             block_table, kv_len, q_start, o, lse, self.ws, stream)
        return o

    def check(self, stream=None):
        """Raises MoeError if a step since the last check met something out of range."""
        moe_check_device_status(self.ws, stream)


class MxLinear:
    """A projection with MXFP4 weights, y = x W^T + bias + residual, its scales laid out in tiles and its
    workspace and output allocated once (torch, on `device`).

    codes [N, K/2] and scales [N, K/32] uint8 as the MXFP4 expert weights have them (or
    `MxLinear.from_weight`); bias [N] fp32 or None. `forward(x, residual)` takes x [T, K] bf16, whose
    rows may lie apart, and residual [T, N] bf16 or None, at most max_tokens rows, and returns
    y [T, N] bf16: `out`, or the layer's own buffer, which the next forward overwrites. Tensors of
    another type, size, layout or device raise ValueError; an `out` that overlaps x, or the residual
    otherwise than as the same tensor, raises MoeError (other columns of one buffer do not overlap).
    """

    def __init__(self, codes, scales, bias=None, max_tokens=4096, device="cuda"):
        import torch
        dev = torch.device(device)
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self._bf16, self._dev = torch.bfloat16, dev
        N, K = codes.shape[0], 2 * codes.shape[1]
        for name, t, dt, shape in (("codes", codes, torch.uint8, (N, K // 2)),
                                   ("scales", scales, torch.uint8, (N, K // 32)),
                                   ("bias", bias, torch.float32, (N,))):
            if t is not None and (t.dtype != dt or tuple(t.shape) != shape or t.device != dev
                                  or not t.is_contiguous()):
                raise ValueError(f"{name}: {t.dtype}, {tuple(t.shape)}, strides {t.stride()} on "
                                 f"{t.device}: packed {dt} {shape} on {dev} is needed")
        self._own(N, K, codes, bias, max_tokens)
        moe_mx_tile_scales(mx_rows(N, K, tiles=True), scales, self.w_scales)

    def _own(self, N, K, codes, bias, max_tokens):
        import torch
        n = moe_mx_linear_workspace_size(mx_shape(max_tokens, N, K))
        if n == 0:
            raise MoeError(-1, "MxLinear", moe_last_error_string())
        self.N, self.K, self.max_tokens = N, K, max_tokens
        self.codes, self.bias = codes, bias
        self.w_scales = torch.empty(moe_mx_scale_bytes(mx_rows(N, K, tiles=True)),
                                    dtype=torch.uint8, device=self._dev)
        self.ws = torch.empty(n, dtype=torch.uint8, device=self._dev)
        self.ws[:4].zero_()
        self.y = torch.empty(max_tokens, N, dtype=torch.bfloat16, device=self._dev)

    @classmethod
    def from_weight(cls, weight, bias=None, max_tokens=4096):
        """The projection of a weight [N, K] in bf16 or fp32 (rows packed), quantised here."""
        import torch
        kind = {torch.bfloat16: "bf16", torch.float32: "f32"}.get(weight.dtype)
        if kind is None or weight.dim() != 2 or not weight.is_contiguous():
            raise ValueError(f"weight: {weight.dtype}, {tuple(weight.shape)}, strides "
                             f"{weight.stride()}: packed [N, K] in bf16 or fp32 is needed")
        N, K = weight.shape
        codes = torch.empty(N, K // 2, dtype=torch.uint8, device=weight.device)
        scales = torch.empty(N, K // 32, dtype=torch.uint8, device=weight.device)
        moe_mx_quantize(mx_rows(N, K, kind), weight, codes, scales)
        return cls(codes, scales, bias, max_tokens, weight.device)

    def _rows_apart(self, name, t, T, n):
        """The distance of the T rows of n packed bf16."""
        if (t.dtype == self._bf16 and t.device == self._dev and t.dim() == 2
                and tuple(t.shape) == (T, n)):
            if t.is_contiguous():
                return n
            if t[0].is_contiguous() and t.stride(0) >= n:
                return t.stride(0)
        raise ValueError(f"{name}: {t.dtype}, {tuple(t.shape)}, strides {t.stride()} on {t.device}: "
                         f"{T} rows of {n} packed bf16 on {self._dev} are needed")

    def forward(self, x, residual=None, out=None, stream=None):
        T = x.shape[0]
        if T > self.max_tokens:
            raise ValueError(f"{T} tokens: the layer was made for {self.max_tokens}")
        y = self.y[:T] if out is None else out
        s = mx_shape(T, self.N, self.K, "bf16", self._rows_apart("x", x, T, self.K),
                     self._rows_apart("out", y, T, self.N),
                     0 if residual is None else self._rows_apart("residual", residual, T, self.N))
        moe_mx_linear(s, x, None, self.codes, self.w_scales, self.bias, residual, y, self.ws, stream)
        return y

    def check(self, stream=None):
        """Raises MoeError if a call since the last check gave up a wait."""
        moe_check_device_status(self.ws, stream)
