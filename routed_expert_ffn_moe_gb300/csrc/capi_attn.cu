// The C ABI of the attention operators (include/moe.h): host-side validation and dispatch.
#include <algorithm>
#include <cmath>

#include "attn.h"
#include "capi.h"

namespace moe {
namespace {

// a stride given in elements of `esz` bytes: the packed one if 0, else a multiple of 16 bytes
// that is at least the packed one
moe_status take_stride(const char* name, int64_t given, int64_t packed, int esz, int64_t* out) {
  *out = given ? given : packed;
  if (*out < packed || *out > (int64_t)1 << 40 || (*out * esz) % 16)
    return fail(MOE_ERR_INVALID_ARG, "%s=%lld not a multiple of 16 bytes of at least %lld elements",
                name, (long long)given, (long long)packed);
  return MOE_OK;
}

moe_status check_attn(const moe_attn_shape* s, AttnDims* a) {
  if (!s) return fail(MOE_ERR_INVALID_ARG, "shape is NULL");
  if (s->T < 0 || s->T > (1 << 24))
    return fail(MOE_ERR_INVALID_ARG, "T=%d not in [0, 2^24]", s->T);
  if (s->B < 0 || s->B > (1 << 20))
    return fail(MOE_ERR_INVALID_ARG, "B=%d not in [0, 2^20]", s->B);
  if (s->D != 64 && s->D != 128)
    return fail(MOE_ERR_UNSUPPORTED, "D=%d: heads are 64 or 128 wide", s->D);
  if (s->Hkv < 1 || s->Hkv > 1024) return fail(MOE_ERR_INVALID_ARG, "Hkv=%d not in [1, 1024]", s->Hkv);
  if (s->Hq < 1 || s->Hq % s->Hkv || s->Hq / s->Hkv > 128)
    return fail(MOE_ERR_INVALID_ARG, "Hq=%d not Hkv=%d times 1 .. 128", s->Hq, s->Hkv);
  if (s->kv_dtype != MOE_KV_BF16 && s->kv_dtype != MOE_KV_FP8_E4M3)
    return fail(MOE_ERR_INVALID_ARG, "kv_dtype=%d unknown", s->kv_dtype);
  if (s->page_size < 1 || s->max_pages < 1 || s->num_pages < 1)
    return fail(MOE_ERR_INVALID_ARG, "page_size=%d, max_pages=%d, num_pages=%d: at least 1 each",
                s->page_size, s->max_pages, s->num_pages);
  if ((int64_t)s->page_size * s->max_pages > (1 << 30))
    return fail(MOE_ERR_INVALID_ARG, "page_size=%d times max_pages=%d is over 2^30", s->page_size,
                s->max_pages);
  if (s->window < 0 || s->n_sink < 0)
    return fail(MOE_ERR_INVALID_ARG, "window=%d, n_sink=%d: not negative", s->window, s->n_sink);
  if (s->rot_dim < 0 || s->rot_dim > s->D || s->rot_dim % 16)
    return fail(MOE_ERR_INVALID_ARG, "rot_dim=%d not a multiple of 16 in [0, D]", s->rot_dim);
  if (s->max_pos < 0) return fail(MOE_ERR_INVALID_ARG, "max_pos=%d is negative", s->max_pos);
  if (!std::isfinite(s->scale) || s->scale < 0.f || !std::isfinite(s->eps) || s->eps < 0.f)
    return fail(MOE_ERR_INVALID_ARG, "scale=%g, eps=%g: finite and not negative", s->scale, s->eps);
  a->T = s->T;
  a->B = s->B;
  a->Hq = s->Hq;
  a->Hkv = s->Hkv;
  a->G = s->Hq / s->Hkv;
  a->D = s->D;
  a->fp8 = s->kv_dtype == MOE_KV_FP8_E4M3;
  a->page_size = s->page_size;
  a->max_pages = s->max_pages;
  a->num_pages = s->num_pages;
  // no place lies beyond those of the table, and sums with limits up to 2^30 fit 32 bits
  const int places = s->page_size * s->max_pages;
  a->window = std::min(s->window, places);
  a->n_sink = s->window ? std::min(s->n_sink, places) : 0;
  a->rot_dim = s->rot_dim;
  a->rot_pairs = s->rot_pairs != 0;
  a->max_pos = s->max_pos;
  a->scale = s->scale > 0.f ? s->scale : 1.0f / std::sqrt((float)s->D);
  a->eps = s->eps;
  a->page_div = fast_div((uint32_t)s->page_size);
  const int64_t q = (int64_t)s->Hq * s->D, kv = (int64_t)s->Hkv * s->D;
  const int esz = a->fp8 ? 1 : 2;
  moe_status st;
  if ((st = take_stride("q_stride", s->q_stride, q, 2, &a->q_stride)) != MOE_OK) return st;
  if ((st = take_stride("k_stride", s->k_stride, kv, 2, &a->k_stride)) != MOE_OK) return st;
  if ((st = take_stride("v_stride", s->v_stride, kv, 2, &a->v_stride)) != MOE_OK) return st;
  if ((st = take_stride("qr_stride", s->qr_stride, q, 2, &a->qr_stride)) != MOE_OK) return st;
  if ((st = take_stride("o_stride", s->o_stride, q, 2, &a->o_stride)) != MOE_OK) return st;
  // the cache: its packed strides, or all three given, in either order of heads and tokens
  const int given = (s->page_stride != 0) + (s->head_stride != 0) + (s->token_stride != 0);
  if (given != 0 && given != 3)
    return fail(MOE_ERR_INVALID_ARG,
                "page_stride, head_stride and token_stride are given together or not at all");
  const int64_t ts = given ? s->token_stride : s->D;
  const int64_t hs = given ? s->head_stride : (int64_t)s->page_size * s->D;
  if ((st = take_stride("token_stride", ts, s->D, esz, &a->token_stride)) != MOE_OK) return st;
  if ((st = take_stride("head_stride", hs, s->D, esz, &a->head_stride)) != MOE_OK) return st;
  return take_stride("page_stride", given ? s->page_stride : kv * s->page_size,
                     kv * s->page_size, esz, &a->page_stride);
}

// the rows that prefill unpacks a cache into: within what a size and a tensor map's strides hold
moe_status check_unpacked(const AttnDims& a) {
  const int64_t row = (int64_t)a.B * a.Hkv * a.D * 4;  // bytes of a place, keys and values
  if (!prefill_reads_pages(a) && row && unpacked_len(a) > ((int64_t)1 << 40) / row)
    return fail(MOE_ERR_INVALID_ARG,
                "B=%d sequences of %lld places, unpacked for prefill, are over 2^40 bytes", a.B,
                (long long)unpacked_len(a));
  return MOE_OK;
}

moe_status check_attn_ws(const AttnDims& a, int prefill, const void* ws, size_t ws_bytes,
                         AttnWs* L) {
  REQUIRE_PTR(ws, 256);
  *L = attn_ws(a, prefill);
  if (ws_bytes < L->total)
    return fail(MOE_ERR_WORKSPACE, "workspace %zu bytes < %zu required", ws_bytes, L->total);
  return MOE_OK;
}

moe_status check_scales(const AttnDims& a, const float* k_scale, const float* v_scale) {
  if (!a.fp8 && (k_scale || v_scale))
    return fail(MOE_ERR_INVALID_ARG, "k_scale/v_scale must be NULL for a bf16 cache");
  if (!aligned(k_scale, 4) || !aligned(v_scale, 4))
    return fail(MOE_ERR_INVALID_ARG, "k_scale/v_scale not 4-byte aligned");
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_attn_workspace_size(const moe_attn_shape* shape, int prefill) {
  AttnDims a;
  if (check_attn(shape, &a) != MOE_OK) return 0;
  if (prefill && check_unpacked(a) != MOE_OK) return 0;
  return attn_ws(a, prefill).total;
}

size_t moe_attn_workspace_zero_bytes(void) { return kAttnZeroBytes; }

moe_status moe_attn_append(const moe_attn_shape* shape, const void* q, const void* k,
                           const void* v, const void* q_norm, const void* k_norm,
                           const float* cos_sin, const int32_t* positions,
                           const int32_t* block_table, const int32_t* kv_len,
                           const int32_t* q_start, const float* k_scale, const float* v_scale,
                           void* q_out, void* k_cache, void* v_cache, void* ws, size_t ws_bytes,
                           void* stream) {
  AttnDims a;
  moe_status st = check_attn(shape, &a);
  if (st != MOE_OK) return st;
  if (!q_start && a.T != a.B)
    return fail(MOE_ERR_INVALID_ARG, "T=%d, B=%d: q_start may be NULL only if T = B", a.T, a.B);
  AttnWs L;
  if ((st = check_attn_ws(a, 0, ws, ws_bytes, &L)) != MOE_OK) return st;
  if (a.T == 0 || a.B == 0) return MOE_OK;
  REQUIRE_PTR(q, 16);
  REQUIRE_PTR(k, 16);
  REQUIRE_PTR(v, 16);
  REQUIRE_PTR(q_out, 16);
  REQUIRE_PTR(k_cache, 16);
  REQUIRE_PTR(v_cache, 16);
  REQUIRE_PTR(block_table, 4);
  REQUIRE_PTR(kv_len, 4);
  if (q_norm && !aligned(q_norm, 16))
    return fail(MOE_ERR_INVALID_ARG, "q_norm not 16-byte aligned");
  if (k_norm && !aligned(k_norm, 16))
    return fail(MOE_ERR_INVALID_ARG, "k_norm not 16-byte aligned");
  if (a.rot_dim) REQUIRE_PTR(cos_sin, 16);
  if (!aligned(positions, 4) || !aligned(q_start, 4))
    return fail(MOE_ERR_INVALID_ARG, "positions/q_start not 4-byte aligned");
  if (q == q_out && a.q_stride != a.qr_stride)
    return fail(MOE_ERR_INVALID_ARG, "q_out is q but qr_stride=%lld is not q_stride=%lld",
                (long long)a.qr_stride, (long long)a.q_stride);
  if ((st = check_scales(a, k_scale, v_scale)) != MOE_OK) return st;
  int* status = reinterpret_cast<int*>(static_cast<char*>(ws) + L.status);
  cudaError_t e = launch_attn_append(a, q, k, v, q_norm, k_norm, cos_sin, positions, block_table,
                                     kv_len, q_start, k_scale, v_scale, q_out, k_cache, v_cache,
                                     status, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : cuda_fail(e, "moe_attn_append launch");
}

moe_status moe_attn_decode(const moe_attn_shape* shape, const void* q, const void* k_cache,
                           const void* v_cache, const float* k_scale, const float* v_scale,
                           const int32_t* block_table, const int32_t* kv_len, void* o, float* lse,
                           void* ws, size_t ws_bytes, void* stream) {
  AttnDims a;
  moe_status st = check_attn(shape, &a);
  if (st != MOE_OK) return st;
  if (a.T != a.B)
    return fail(MOE_ERR_INVALID_ARG, "T=%d, B=%d: decode takes one token per sequence", a.T, a.B);
  AttnWs L;
  if ((st = check_attn_ws(a, 0, ws, ws_bytes, &L)) != MOE_OK) return st;
  if (a.B == 0) return MOE_OK;
  REQUIRE_PTR(q, 16);
  REQUIRE_PTR(k_cache, 16);
  REQUIRE_PTR(v_cache, 16);
  REQUIRE_PTR(block_table, 4);
  REQUIRE_PTR(kv_len, 4);
  REQUIRE_PTR(o, 16);
  if (!aligned(lse, 4)) return fail(MOE_ERR_INVALID_ARG, "lse not 4-byte aligned");
  if ((st = check_scales(a, k_scale, v_scale)) != MOE_OK) return st;
  cudaError_t e = launch_attn_decode(a, q, k_cache, v_cache, k_scale, v_scale, block_table,
                                     kv_len, o, lse, static_cast<char*>(ws), L,
                                     static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : cuda_fail(e, "moe_attn_decode launch");
}

moe_status moe_attn_prefill(const moe_attn_shape* shape, const void* q, const void* k_cache,
                            const void* v_cache, const float* k_scale, const float* v_scale,
                            const int32_t* block_table, const int32_t* kv_len,
                            const int32_t* q_start, void* o, float* lse, void* ws,
                            size_t ws_bytes, void* stream) {
  AttnDims a;
  moe_status st = check_attn(shape, &a);
  if (st != MOE_OK) return st;
  if ((int64_t)a.T * a.Hkv >= (int64_t)1 << 30)
    return fail(MOE_ERR_INVALID_ARG, "T=%d times Hkv=%d is over 2^30", a.T, a.Hkv);
  if ((st = check_unpacked(a)) != MOE_OK) return st;
  AttnWs L;
  if ((st = check_attn_ws(a, 1, ws, ws_bytes, &L)) != MOE_OK) return st;
  if (a.T == 0 || a.B == 0) return MOE_OK;
  REQUIRE_PTR(q, 16);
  REQUIRE_PTR(k_cache, 16);
  REQUIRE_PTR(v_cache, 16);
  REQUIRE_PTR(block_table, 4);
  REQUIRE_PTR(kv_len, 4);
  REQUIRE_PTR(q_start, 4);
  REQUIRE_PTR(o, 16);
  if (!aligned(lse, 4)) return fail(MOE_ERR_INVALID_ARG, "lse not 4-byte aligned");
  if ((st = check_scales(a, k_scale, v_scale)) != MOE_OK) return st;
  cudaError_t e = launch_attn_prefill(a, q, k_cache, v_cache, k_scale, v_scale, block_table,
                                      kv_len, q_start, o, lse, static_cast<char*>(ws), L,
                                      static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : cuda_fail(e, "moe_attn_prefill launch");
}

}  // extern "C"
