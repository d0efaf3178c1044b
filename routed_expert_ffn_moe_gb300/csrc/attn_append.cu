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
// Layout: one block per token (and, for small batches, per slice of its heads). D/8 lanes hold a
// head, eight consecutive elements (16 bytes) each: the norm is a butterfly over those lanes, a
// pair of neighbours turns inside a lane, and a pair (i, i + rot/2) is one shuffle apart. Each
// lane group keeps its eight cosines and sines in registers across the heads that it takes.
#include "attn.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

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

template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads) k_attn_append(const AppendParams p) {
  constexpr int LPH = D / 8;               // lanes of a head
  constexpr int GROUPS = kThreads / LPH;   // heads in flight in a block
  constexpr int kBatch = 4;                // heads whose loads a lane group issues together
  const AttnDims& a = p.a;
  const int t = (int)blockIdx.x;
  const int sub = (int)threadIdx.x % LPH;  // this lane's eight elements of a head
  const int grp = (int)threadIdx.x / LPH;
  pdl_wait_then_release();

  // The token's sequence: the number of sequences that end at or before it.
  int b = t, n = 1, i = 0;
  if (p.q_start) {
    int cnt = 0;
    for (int s = (int)threadIdx.x; s - (int)threadIdx.x < a.B; s += kThreads) {
      const int here = __syncthreads_count(s < a.B && __ldg(p.q_start + s + 1) <= t);
      cnt += here;
      if (here < kThreads) break;
    }
    b = cnt;
    if (b < a.B) {
      const int q0 = __ldg(p.q_start + b);
      n = __ldg(p.q_start + b + 1) - q0;
      i = t - q0;
    }
  }
  // Its place in the cache and its rotary position; whatever is out of range is not touched.
  int64_t slot = -1;
  int pos = 0;
  bool live = b < a.B && i >= 0, bad = i < 0;  // rows from q_start[B] on are padding too
  if (live) {
    const int len = __ldg(p.kv_len + b);
    const int place = len - n + i;
    live = place >= 0;  // a negative place is padding
    if (live) {
      const uint32_t pg = div_fast((uint32_t)place, a.page_div);
      if (pg >= (uint32_t)a.max_pages) {
        bad = true;
      } else {
        const int page = __ldg(p.block_table + (int64_t)b * a.max_pages + pg);
        if ((uint32_t)page >= (uint32_t)a.num_pages)
          bad = true;
        else
          slot = (int64_t)page * a.page_stride +
                 (int64_t)(place - (int)pg * a.page_size) * a.token_stride;
      }
      pos = p.positions ? __ldg(p.positions + t) : place;
      if (a.rot_dim && (uint32_t)pos >= (uint32_t)a.max_pos) {
        bad = true;
        live = false;
      }
    }
  }
  if (bad && threadIdx.x == 0) record_error(p.status, MOE_ERR_DEVICE_BOUNDS);

  // Eight cosines and sines a lane, for the elements it holds (0: not rotated).
  const int half = a.rot_dim >> 1;
  const bool turns = live && sub * 8 < a.rot_dim;
  float c[8], s[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) c[e] = 1.f, s[e] = 0.f;
  int partner = sub;   // lane that holds the other halves of this lane's pairs
  if (turns) {
    const float* row = p.cos_sin + (int64_t)pos * a.rot_dim;
    if (a.rot_pairs) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        c[2 * e] = c[2 * e + 1] = __ldg(row + sub * 4 + e);
        s[2 * e + 1] = __ldg(row + half + sub * 4 + e);
        s[2 * e] = -s[2 * e + 1];
      }
    } else {
      const bool first = sub * 8 < half;
      const int at = first ? sub * 8 : sub * 8 - half;
      partner = first ? sub + (half >> 3) : sub - (half >> 3);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        c[e] = __ldg(row + at + e);
        const float sn = __ldg(row + half + at + e);
        s[e] = first ? -sn : sn;
      }
    }
  }
  const int src_lane = (((int)threadIdx.x & 31) / LPH) * LPH + partner;

  const int heads = a.Hq + 2 * a.Hkv;
  const int per = ((heads + (int)gridDim.y - 1) / (int)gridDim.y);
  const int h0 = (int)blockIdx.y * per, h1 = min(heads, h0 + per);
  // rounds of the whole block, so that every lane of a warp reaches the shuffles
  for (int base = h0; base < h1; base += kBatch * GROUPS) {
    uint4 u[kBatch];
#pragma unroll
    for (int r = 0; r < kBatch; ++r) {
      const int h = base + r * GROUPS + grp;
      const uint16_t* src = p.q + (int64_t)t * a.q_stride + (int64_t)h * D;
      if (h >= a.Hq + a.Hkv)
        src = p.v + (int64_t)t * a.v_stride + (int64_t)(h - a.Hq - a.Hkv) * D;
      else if (h >= a.Hq)
        src = p.k + (int64_t)t * a.k_stride + (int64_t)(h - a.Hq) * D;
      u[r] = make_uint4(0, 0, 0, 0);
      if (h < h1) u[r] = *reinterpret_cast<const uint4*>(src + sub * 8);
    }
#pragma unroll
    for (int r = 0; r < kBatch; ++r) {
      const int h = base + r * GROUPS + grp;
      if (base + r * GROUPS >= h1) break;  // the same for the whole block
      float x[8];
      unpack8(u[r], x);
      const bool is_v = h >= a.Hq + a.Hkv, is_q = h < a.Hq;
      const uint16_t* w = is_q ? p.q_norm : p.k_norm;
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
      for (int o = LPH / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (w && !is_v) {
        const float inv = rsqrtf(ss * (1.0f / D) + a.eps);
        float wf[8];
        unpack8(ldg_u4(w + sub * 8), wf);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] * inv * wf[e];
      }
      float y[8];
      if (a.rot_pairs) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = x[e ^ 1];
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = __shfl_sync(0xffffffffu, x[e], src_lane);
      }
      if (!is_v && turns) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = fmaf(x[e], c[e], y[e] * s[e]);
      }
      if (h >= h1) continue;
      if (is_q) {
        const uint4 out = live ? pack8_bf16(x) : make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4*>(p.q_out + (int64_t)t * a.qr_stride + (int64_t)h * D + sub * 8) =
            out;
      } else if (slot >= 0 && live) {
        const int hk = is_v ? h - a.Hq - a.Hkv : h - a.Hq;
        uint8_t* cache = is_v ? p.v_cache : p.k_cache;
        const int64_t at = slot + (int64_t)hk * a.head_stride + sub * 8;
        if (FP8) {
          const float* sc = is_v ? p.v_scale : p.k_scale;
          *reinterpret_cast<uint2*>(cache + at) = pack8_e4m3(x, sc ? __ldg(sc + hk) : 1.f);
        } else {
          *reinterpret_cast<uint4*>(cache + 2 * at) = pack8_bf16(x);
        }
      }
    }
  }
}

template <int D, bool FP8>
cudaError_t launch(const AppendParams& p, cudaStream_t st) {
  // Below two blocks an SM the heads of a token are spread over blocks, one round each.
  const int rounds = (p.a.Hq + 2 * p.a.Hkv + kThreads / (D / 8) - 1) / (kThreads / (D / 8));
  const int ny = p.a.T < 2 * num_sms() ? rounds : 1;
  count_launches(1);
  return launch_pdl(k_attn_append<D, FP8>, dim3((unsigned)p.a.T, (unsigned)ny), dim3(kThreads), 0,
                    st, p);
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
