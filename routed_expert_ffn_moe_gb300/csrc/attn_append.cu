// Per-head norms, position rotation and append to the paged cache, in one pass.
//
// For a head vector x of D elements (a query head, or a key head):
//   y = x / sqrt(mean(x^2) + eps) * w          (if a norm weight is given)
//   (y_a, y_b) <- (y_a c - y_b s, y_b c + y_a s) for each rotated pair, c and s from the table
// in fp32, rounded once: to bf16 (queries, bf16 caches) or to E4M3 of y / scale. Values are only
// copied or converted.
//
// What bounds it: HBM. A token reads (Hq + 2 Hkv) D bf16 and writes as many elements; nothing is
// read twice but the norm weights and the token's row of the table (both from L1/L2).
//
// Layout: D/8 lanes hold a head, eight consecutive elements (16 bytes) each: the norm is a
// butterfly over those lanes, a pair of neighbours turns inside a lane, and the other half of a
// pair (i, i + rot/2) is fetched from its lane as packed bf16. With coefficients that a lane forms
// once per token and kind of head, A = w c and S = +-w' s (w' and s of the other element of the
// pair), a head is  y = inv (x A + x' S); where nothing turns x' and S are zeros, so that an
// infinity passes through (0 times one would be a NaN).
// A lane group belongs to one token and takes its heads in turn, a batch of loads ahead; it finds
// its token's sequence, place and page by itself while the first batch is on its way. Nothing
// synchronises a block.
#include "attn.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;  // heads of a batch
// Lanes (tokens x heads x D / 8) of a small step. Small kernel against large, us, bf16, query + key
// heads: of 64, 4+1, 1024 tokens 2.6 against 4.2, 4096 4.7 against 4.2; 64+8, 256 tokens 3.4 against
// 4.2, 1024 9.3 against 8.9. Of 128, 4+1, 1024 tokens 3.5 against 4.3, 2048 4.9 against 4.4; 64+8, 64
// tokens 2.8 against 4.3, 256 5.7 against 6.3, 1024 20.5 against 14.4.
constexpr int64_t kSmallLanes = 5 << 16;

struct AppendParams {
  AttnDims a;
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  const uint16_t* q_norm;
  const uint16_t* k_norm;
  const float* cos_sin;
  const int32_t* positions;
  const int32_t* block_table;
  const int32_t* kv_len;
  const int32_t* q_start;
  const float* k_scale;
  const float* v_scale;
  uint16_t* q_out;
  uint8_t* k_cache;
  uint8_t* v_cache;
  int* status;
  int groups;  // large: lane groups of a token in a block (a power of two)
  FastDiv heads_div;  // small: by the heads of a token, of all kinds
};

__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  x[0] = bf16_lo(u.x); x[1] = bf16_hi(u.x);
  x[2] = bf16_lo(u.y); x[3] = bf16_hi(u.y);
  x[4] = bf16_lo(u.z); x[5] = bf16_hi(u.z);
  x[6] = bf16_lo(u.w); x[7] = bf16_hi(u.w);
}

__device__ __forceinline__ uint4 pack8_bf16(const float (&x)[8]) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                    pack_bf16(x[6], x[7]));
}

// e4m3(x / scale), nearest even, saturating; a NaN stays one
__device__ __forceinline__ uint2 pack8_e4m3(const float (&x)[8], float scale) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(lo) : "f"(__fdiv_rn(x[4 * i + 1], scale)), "f"(__fdiv_rn(x[4 * i], scale)));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(hi) : "f"(__fdiv_rn(x[4 * i + 3], scale)), "f"(__fdiv_rn(x[4 * i + 2], scale)));
    w[i] = (uint32_t)lo | ((uint32_t)hi << 16);
  }
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ uint64_t pair_of(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void split(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Where a token's keys and values go, and how its heads turn.
struct Place {
  int64_t slot;  // its row in the cache, of key head 0 (-1: nothing is written)
  int pos;       // its rotary position
  bool live;     // false: padding, or out of range: its queries are zeros
};

// Found by the LPH lanes of a group together; every group of a warp takes part.
template <int LPH>
__device__ __forceinline__ Place find_place(const AppendParams& p, int tok) {
  const AttnDims& a = p.a;
  const int sub = (int)threadIdx.x % LPH, lane0 = ((int)threadIdx.x & 31) - sub;
  const int t = min(tok, a.T - 1);
  int b = t, q0 = t, q1 = t + 1, len = 0;
  if (p.q_start) {
    // as many tokens as sequences: most likely one each
    bool mine = false;
    if (a.T == a.B) {
      q0 = __ldg(p.q_start + t);
      q1 = __ldg(p.q_start + t + 1);
      len = __ldg(p.kv_len + t);
      mine = q0 == t && q1 == t + 1;
    }
    if (__any_sync(0xffffffffu, !mine)) {
      // the number of sequences that end at or before the token, by LPH probes a round
      b = 0;
      for (int left = a.B; left > 0;) {  // it is b .. b + left; the same rounds for everyone
        const int gap = (left + LPH - 1) / LPH, s = b + (sub + 1) * gap - 1;
        const bool past = s < a.B && __ldg(p.q_start + s + 1) <= t;
        const unsigned votes = __ballot_sync(0xffffffffu, past);
        b += __popc((votes >> lane0) & (LPH == 32 ? 0xffffffffu : (1u << LPH) - 1)) * gap;
        left = gap - 1;
      }
      b = min(b, a.B);
      if (b < a.B) {
        q0 = __ldg(p.q_start + b);
        q1 = __ldg(p.q_start + b + 1);
        len = __ldg(p.kv_len + b);
      }
    }
  } else {
    len = __ldg(p.kv_len + b);
  }
  Place at{-1, 0, tok < a.T && b < a.B && q0 <= t};  // rows from q_start[B] on are padding
  bool bad = b < a.B && q0 > t;
  const int place = len - q1 + t;  // negative: padding
  at.live = at.live && place >= 0;
  if (at.live) {
    const uint32_t pg = div_fast((uint32_t)place, a.page_div);
    at.pos = p.positions ? __ldg(p.positions + t) : place;
    if (pg >= (uint32_t)a.max_pages) {
      bad = true;
    } else {
      const int page = __ldg(p.block_table + (int64_t)b * a.max_pages + pg);
      if ((uint32_t)page >= (uint32_t)a.num_pages)
        bad = true;
      else
        at.slot = (int64_t)page * a.page_stride +
                  (int64_t)(place - (int)pg * a.page_size) * a.token_stride;
    }
    if (a.rot_dim && (uint32_t)at.pos >= (uint32_t)a.max_pos) {
      bad = true;
      at.live = false;
      at.slot = -1;
    }
  }
  if (bad && tok < a.T && sub == 0) record_error(p.status, MOE_ERR_DEVICE_BOUNDS);
  return at;
}

// A lane's coefficients for one kind of head, and the lane (of its group) that holds the other
// halves of its pairs.
struct Turn {
  uint64_t A[4], S[4];
  int partner;
  uint32_t other;  // ones where the lane's elements turn: a mask of the other halves
};

template <int LPH>
__device__ __forceinline__ void coefficients(const AppendParams& p, const Place& at,
                                             const uint16_t* w, Turn& k) {
  const AttnDims& a = p.a;
  const int sub = (int)threadIdx.x % LPH, half = a.rot_dim >> 1;
  const bool turns = at.live && sub * 8 < a.rot_dim, first = sub * 8 < half;
  k.other = turns ? 0xffffffffu : 0u;
  k.partner = !turns || a.rot_pairs ? sub : first ? sub + (half >> 3) : sub - (half >> 3);
  float own[8], other[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) own[e] = other[e] = 1.f;
  if (w) {
    unpack8(ldg_u4(w + sub * 8), own);
    unpack8(ldg_u4(w + k.partner * 8), other);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    k.A[e] = pair_of(own[2 * e], own[2 * e + 1]);
    k.S[e] = pair_of(-0.f, -0.f);  // x A + 0 S is x A of either sign
  }
  if (!turns) return;
  const float* cs = p.cos_sin + (int64_t)at.pos * a.rot_dim +
                    (a.rot_pairs ? sub * 4 : first ? sub * 8 : sub * 8 - half);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (a.rot_pairs) {  // elements 2e, 2e + 1 turn with each other
      const float c = __ldg(cs + e), s = __ldg(cs + half + e);
      k.A[e] = mul2(k.A[e], pair_of(c, c));
      k.S[e] = pair_of(other[2 * e + 1] * -s, other[2 * e] * s);
    } else {
      const float2 c = __ldg(reinterpret_cast<const float2*>(cs) + e);
      const float2 s = __ldg(reinterpret_cast<const float2*>(cs + half) + e);
      const float sign = first ? -1.f : 1.f;
      k.A[e] = mul2(k.A[e], pair_of(c.x, c.y));
      k.S[e] = pair_of(other[2 * e] * (sign * s.x), other[2 * e + 1] * (sign * s.y));
    }
  }
}

// A head's eight elements, normed (if `norm`; `any`: if any head of the warp may be) and turned.
template <int LPH>
__device__ __forceinline__ void turn_head(const AttnDims& a, const Turn& k, bool any, bool norm,
                                          const uint4& u, float (&z)[8]) {
  const int lane0 = ((int)threadIdx.x & 31) - (int)threadIdx.x % LPH;
  const uint32_t in[4] = {u.x, u.y, u.z, u.w};
  uint64_t x[4], y[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[e] = pair_of(bf16_lo(in[e]), bf16_hi(in[e]));
    if (a.rot_pairs) {
      const uint32_t o = in[e] & k.other;
      y[e] = pair_of(bf16_hi(o), bf16_lo(o));
    } else {
      const uint32_t o = __shfl_sync(0xffffffffu, in[e], lane0 + k.partner) & k.other;
      y[e] = pair_of(bf16_lo(o), bf16_hi(o));
    }
  }
  float inv = 1.f;
  if (any) {
    uint64_t ss = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) ss = fma2(x[e], x[e], ss);
    float lo, hi;
    split(ss, lo, hi);
    lo += hi;
#pragma unroll
    for (int o = LPH / 2; o; o >>= 1) lo += __shfl_xor_sync(0xffffffffu, lo, o);
    if (norm) inv = rsqrtf(lo * (1.0f / (8 * LPH)) + a.eps);
  }
  const uint64_t inv2 = pair_of(inv, inv);
#pragma unroll
  for (int e = 0; e < 4; ++e)
    split(mul2(fma2(x[e], k.A[e], mul2(y[e], k.S[e])), inv2), z[2 * e], z[2 * e + 1]);
}

template <bool FP8>
__device__ __forceinline__ void store_cache(const AppendParams& p, uint8_t* cache,
                                            const float* scale, int64_t slot, int h, int elem,
                                            const float (&z)[8]) {
  if (slot < 0) return;
  const int64_t at = slot + (int64_t)h * p.a.head_stride + elem;
  if (FP8)
    *reinterpret_cast<uint2*>(cache + at) = pack8_e4m3(z, scale ? __ldg(scale + h) : 1.f);
  else
    *reinterpret_cast<uint4*>(cache + 2 * at) = pack8_bf16(z);
}

// Large steps: a lane group takes the heads of its token in turn, `groups` of them to a token. 16245
// tokens of 64 + 8 + 8 heads of 128: 107 us, 0.92 of the measured copy rate; 4096, 34 us, 0.73; over
// E4M3, 16384 tokens 119 us, 0.80.
template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads, 3) k_attn_append(const AppendParams p) {
  constexpr int LPH = D / 8, GROUPS = kThreads / LPH;
  const AttnDims& a = p.a;
  const int sub = (int)threadIdx.x % LPH, grp = (int)threadIdx.x / LPH;
  const int tok = (int)blockIdx.x * (GROUPS / p.groups) + grp / p.groups;
  const int t = min(tok, a.T - 1), h0 = grp % p.groups, step = p.groups;
  pdl_wait_then_release();

  // a batch of heads h, h + step, ... of `n` from a row
  const auto fetch = [&](const uint16_t* row, int h, int n, uint4 (&u)[kBatch]) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      u[i] = make_uint4(0, 0, 0, 0);
      if (h + i * step < n) u[i] = *reinterpret_cast<const uint4*>(row + (int64_t)(h + i * step) * D);
    }
  };
  const uint16_t* q_row = p.q + (int64_t)t * a.q_stride + sub * 8;
  const uint16_t* k_row = p.k + (int64_t)t * a.k_stride + sub * 8;
  const uint16_t* v_row = p.v + (int64_t)t * a.v_stride + sub * 8;
  uint4 u[kBatch];
  fetch(q_row, h0, a.Hq, u);
  const Place at = find_place<LPH>(p, tok);

  // the last batch of a kind asks for the first of the next kind
  const auto turned = [&](const uint16_t* row, int heads, const uint16_t* w, const uint16_t* then,
                          const auto& put) {
    Turn k;
    coefficients<LPH>(p, at, w, k);
    for (int base = 0; base < heads; base += kBatch * step) {  // the same rounds for everyone
      uint4 next[kBatch];
      if (base + kBatch * step < heads)
        fetch(row, base + kBatch * step + h0, heads, next);
      else
        fetch(then, h0, a.Hkv, next);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (base + i * step >= heads) break;  // for the whole block
        float z[8];
        turn_head<LPH>(a, k, w != nullptr, w != nullptr, u[i], z);
        const int h = base + i * step + h0;
        if (h < heads && tok < a.T) put(h, z);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) u[i] = next[i];
    }
  };
  turned(q_row, a.Hq, p.q_norm, k_row, [&](int h, const float (&z)[8]) {
    *reinterpret_cast<uint4*>(p.q_out + (int64_t)t * a.qr_stride + (int64_t)h * D + sub * 8) =
        at.live ? pack8_bf16(z) : make_uint4(0, 0, 0, 0);
  });
  turned(k_row, a.Hkv, p.k_norm, v_row, [&](int h, const float (&z)[8]) {
    store_cache<FP8>(p, p.k_cache, p.k_scale, at.slot, h, sub * 8, z);
  });
  for (int h = h0; h < a.Hkv; h += kBatch * step) {
    if (h != h0) fetch(v_row, h, a.Hkv, u);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (h + i * step >= a.Hkv) break;
      float z[8];
      unpack8(u[i], z);
      store_cache<FP8>(p, p.v_cache, p.v_scale, at.slot, h + i * step, sub * 8, z);
    }
  }
}

// Small steps: one head to a lane group, tokens and heads in a row. Short code, many blocks: such a
// step is the latency of its chain of look-ups. 1 token of 32 + 8 + 8 heads of 128: 2.3 us; 256 of 56 +
// 8 + 8, E4M3: 5.9 us.
template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads, 5) k_attn_append_small(const AppendParams p) {
  constexpr int LPH = D / 8, GROUPS = kThreads / LPH;
  const AttnDims& a = p.a;
  const int sub = (int)threadIdx.x % LPH, heads = a.Hq + 2 * a.Hkv;
  const uint32_t row = blockIdx.x * GROUPS + threadIdx.x / LPH;
  const int tok = (int)div_fast(row, p.heads_div), h = (int)row - tok * heads, t = min(tok, a.T - 1);
  const bool is_q = h < a.Hq, is_v = h >= a.Hq + a.Hkv;
  const int hk = is_q ? h : is_v ? h - a.Hq - a.Hkv : h - a.Hq;  // among its kind
  const uint16_t* src = is_q   ? p.q + (int64_t)t * a.q_stride
                        : is_v ? p.v + (int64_t)t * a.v_stride
                               : p.k + (int64_t)t * a.k_stride;
  const uint16_t* w = is_v ? nullptr : is_q ? p.q_norm : p.k_norm;
  pdl_wait_then_release();
  const uint4 u = *reinterpret_cast<const uint4*>(src + (int64_t)hk * D + sub * 8);
  const Place at = find_place<LPH>(p, tok);
  Turn k;
  coefficients<LPH>(p, at, w, k);
  float z[8];
  // a warp holds several heads, of any kinds: the lanes exchange for all of them
  turn_head<LPH>(a, k, p.q_norm != nullptr || p.k_norm != nullptr, w != nullptr, u, z);
  if (tok >= a.T) return;
  if (is_q) {
    *reinterpret_cast<uint4*>(p.q_out + (int64_t)t * a.qr_stride + (int64_t)h * D + sub * 8) =
        at.live ? pack8_bf16(z) : make_uint4(0, 0, 0, 0);
  } else if (is_v) {
    unpack8(u, z);
    store_cache<FP8>(p, p.v_cache, p.v_scale, at.slot, hk, sub * 8, z);
  } else {
    store_cache<FP8>(p, p.k_cache, p.k_scale, at.slot, hk, sub * 8, z);
  }
}

template <int D, bool FP8>
cudaError_t launch(AppendParams& p, cudaStream_t st) {
  constexpr int GROUPS = kThreads / (D / 8);
  const int heads = p.a.Hq + 2 * p.a.Hkv;
  const int64_t rows = (int64_t)p.a.T * heads;
  count_launches(1);
  if (rows * (D / 8) <= kSmallLanes) {
    p.heads_div = fast_div((uint32_t)heads);
    return launch_pdl(k_attn_append_small<D, FP8>, dim3((unsigned)((rows + GROUPS - 1) / GROUPS)),
                      dim3(kThreads), 0, st, p);
  }
  // Fewer groups a token mean fewer look-ups and more heads a group: no more groups than batches of
  // query heads; 16 query heads a group as long as that fills the SMs' places (three blocks each);
  // and more where the blocks would fill them eight times over. 64 + 8 heads of 128, 4096 tokens,
  // 16, 8, 4 groups: 54.0, 38.4, 34.5 us; 16384 tokens, 4, 2, 1: 112.2, 109.2, 115.5. 14 + 2 heads of 64,
  // 4096 tokens, 32, 2: 35.6, 7.8.
  p.groups = GROUPS;
  const auto blocks = [&] { return (int64_t)p.a.T * p.groups / GROUPS; };
  while (p.groups > 1 && (p.groups * kBatch > p.a.Hq || blocks() > 24 * num_sms() ||
                          (p.groups * 8 >= p.a.Hq && blocks() >= 6 * num_sms())))
    p.groups >>= 1;
  const int per_block = GROUPS / p.groups;
  return launch_pdl(k_attn_append<D, FP8>, dim3((unsigned)((p.a.T + per_block - 1) / per_block)),
                    dim3(kThreads), 0, st, p);
}

}  // namespace

cudaError_t launch_attn_append(const AttnDims& a, const void* q, const void* k, const void* v,
                               const void* q_norm, const void* k_norm, const float* cos_sin,
                               const int32_t* positions, const int32_t* block_table,
                               const int32_t* kv_len, const int32_t* q_start,
                               const float* k_scale, const float* v_scale, void* q_out,
                               void* k_cache, void* v_cache, int* status, cudaStream_t st) {
  AppendParams p{};
  p.a = a;
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.q_norm = static_cast<const uint16_t*>(q_norm);
  p.k_norm = static_cast<const uint16_t*>(k_norm);
  p.cos_sin = cos_sin;
  p.positions = positions;
  p.block_table = block_table;
  p.kv_len = kv_len;
  p.q_start = q_start;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.q_out = static_cast<uint16_t*>(q_out);
  p.k_cache = static_cast<uint8_t*>(k_cache);
  p.v_cache = static_cast<uint8_t*>(v_cache);
  p.status = status;
  if (a.D == 64) return a.fp8 ? launch<64, true>(p, st) : launch<64, false>(p, st);
  return a.fp8 ? launch<128, true>(p, st) : launch<128, false>(p, st);
}

}  // namespace moe
