// Internal interface of the attention operators: resolved dimensions, workspace, launchers.
#pragma once

#include "internal.h"

namespace moe {

// moe_attn_shape with every default filled in
struct AttnDims {
  int T, B, Hq, Hkv, G, D;
  int fp8;
  int page_size, max_pages, num_pages;
  int window, n_sink;  // window 0: none (n_sink then 0)
  int rot_dim, rot_pairs, max_pos;
  float scale, eps;
  int64_t q_stride, k_stride, v_stride, qr_stride, o_stride;
  int64_t page_stride, head_stride, token_stride;
  FastDiv page_div;
};

// ---- workspace -----------------------------------------------------------------------------
//   status    int32[64]               device error code (first error wins)
//   parts     f32 [2 * ctas][16][D]   decode: unnormalised outputs of the items that span blocks,
//                                     two a block
//   ml        f32 [2 * ctas][16][2]   decode: their running maxima and sums
//   prefill_parts  f32 [blocks][2][2 * 128][D]   prefill: the same of the units that runs cut
//   prefill_ml     f32 [blocks][2][2 * 128][2]
//   prefill_cuts   [blocks]           prefill: where each run begins
//   unpacked  bf16 [2][B][Hkv][Lp][D] prefill over a cache that its tiles cannot read as it lies:
//                                     keys, then values, each sequence in a row; Lp is
//                                     max_pages * page_size rounded up to a tile
constexpr int kAttnMaxCtas = 512;    // blocks of a decode call, at most
constexpr int kPrefillMaxCtas = 160; // blocks of a prefill call, at most
constexpr size_t kPrefillCutBytes = 64;
constexpr size_t kAttnZeroBytes = 256;  // the status words
constexpr int kDecodeRows = 16;      // query heads of one decode item

struct AttnWs {
  size_t status, parts, ml, prefill_parts, prefill_ml, prefill_cuts, unpacked, total;
};

constexpr int kPrefillKeys = 128;  // the unpacked rows are made in runs of so many places

// Prefill tiles are read by TMA in boxes of one page each: bf16 pages of a multiple of 16 tokens.
// Other caches are unpacked first: E4M3 because the products take bf16, odd pages because a box is
// whole 8-row atoms of the swizzle, and pages of 8 because eight boxes a tile take longer than the
// tile (2048 tokens over 16384 places of 64 heads of 128, 1275 us in place against 682, 8 prompts of
// 1500, 390 against 273, both with an earlier tile loop). In place against unpacked now, us, pages of 16
// and 32: 2048 over 16384, 648 and 648 against 671; 8 x 1500, 241 and 238 against 264; 16 tokens over
// 16384, 42 and 40 against 67.
inline bool prefill_reads_pages(const AttnDims& a) { return !a.fp8 && a.page_size % 16 == 0; }

inline int64_t unpacked_len(const AttnDims& a) {
  const int64_t n = (int64_t)a.max_pages * a.page_size;
  return (n + kPrefillKeys - 1) / kPrefillKeys * kPrefillKeys;
}

inline AttnWs attn_ws(const AttnDims& a, int prefill) {
  AttnWs L{};
  size_t off = 0;
  auto take = [&](size_t bytes) { size_t at = off; off = align_up(off + bytes, 256); return at; };
  L.status = take(256);
  L.parts = take(2 * (size_t)kAttnMaxCtas * kDecodeRows * a.D * 4);
  L.ml = take(2 * (size_t)kAttnMaxCtas * kDecodeRows * 8);
  const size_t rows = prefill ? (size_t)kPrefillMaxCtas * 2 * 2 * 128 : 0;
  L.prefill_parts = take(rows * a.D * 4);
  L.prefill_ml = take(rows * 8);
  L.prefill_cuts = take(prefill ? kPrefillMaxCtas * kPrefillCutBytes : 0);
  const bool unpack = prefill && !prefill_reads_pages(a);
  L.unpacked = take(unpack ? 4 * (size_t)a.B * a.Hkv * unpacked_len(a) * a.D : 0);
  L.total = off;
  return L;
}

// ---- launchers -----------------------------------------------------------------------------
cudaError_t launch_attn_append(const AttnDims& a, const void* q, const void* k, const void* v,
                               const void* q_norm, const void* k_norm, const float* cos_sin,
                               const int32_t* positions, const int32_t* block_table,
                               const int32_t* kv_len, const int32_t* q_start,
                               const float* k_scale, const float* v_scale, void* q_out,
                               void* k_cache, void* v_cache, int* status, cudaStream_t st);
cudaError_t launch_attn_decode(const AttnDims& a, const void* q, const void* k_cache,
                               const void* v_cache, const float* k_scale, const float* v_scale,
                               const int32_t* block_table, const int32_t* kv_len, void* o,
                               float* lse, char* ws, const AttnWs& L, cudaStream_t st);

cudaError_t launch_attn_prefill(const AttnDims& a, const void* q, const void* k_cache,
                                const void* v_cache, const float* k_scale, const float* v_scale,
                                const int32_t* block_table, const int32_t* kv_len,
                                const int32_t* q_start, void* o, float* lse, char* ws,
                                const AttnWs& L, cudaStream_t st);

#ifdef __CUDACC__
__device__ __forceinline__ uint32_t div_fast(uint32_t n, const FastDiv& f) {
  return (uint32_t)(((uint64_t)n * f.m) >> f.p);
}

// two fp32 -> packed bf16 (lo in the low half), round to nearest even
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
#endif

}  // namespace moe
