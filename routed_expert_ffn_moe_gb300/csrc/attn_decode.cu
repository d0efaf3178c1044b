// Attention of one new token per sequence over the paged cache.
//
//   s_j = scale q.k_j over the visible places j,  o = sum_j e^(s_j - m) v_j / l,
//   m = max_j s_j,  l = sum_j e^(s_j - m),  lse = m + ln l
//
// What bounds it: HBM. Every visible key and value is read once, 2 G multiply-adds an element,
// far below the tensor cores' rate even padded to 16 query heads.
//
// Work split. An item is one sequence, one key head and up to 16 of its query heads; a unit is
// one tile of an item's visible keys (64, or 128 of E4M3). All units of the batch in a row are cut
// into equal runs, one per block of a grid that fills the SMs, whatever the lengths are: a
// block ends one item, does some whole ones and begins another. An item that spans blocks leaves
// one partial (m, l, unnormalised o) per block, and the block that arrives last joins them in
// block order, so the result does not depend on timing.
//
// Inside a block every warp has its own 16 (32) keys of each tile and its own ring of
// cp.async stages: it fetches the page of each key, copies the rows (zeros for places that are
// not visible: what the cache holds there never enters a product), and runs the running softmax
// on m16n8k16 MMAs, the 16 rows being query heads. Nothing synchronises the warps until an
// item ends, when they merge through the stage that was just consumed.
//
// Probabilities of a bf16 cache enter the product with v as two bf16 terms (2^-16 relative): the
// tensor cores have room, and one term alone would be the largest error of the result.
//
// E4M3 codes enter the MMAs as f16 (exactly). The queries become f16 too, each row times the
// power of two that brings its largest element to [2^14, 2^15), taken back in the scores'
// scale: elements above 2^-28 of the row's largest are exact. An 8-bit row is read in 16-bit
// pairs, which permutes the contraction index of q.k (the queries are loaded in the same order)
// and the columns of v (stored back in place).
#include "attn.h"
#include "sm100_ptx.cuh"

namespace moe {
namespace {

using namespace ptx;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;

struct DecodeParams {
  AttnDims a;
  const uint16_t* q;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const float* k_scale;
  const float* v_scale;
  const int32_t* block_table;
  const int32_t* kv_len;
  uint16_t* o;
  float* lse;
  int* status;
  int* counters;
  float* parts;
  float2* ml;
  int rt;  // items of a key head: ceil(G / 16)
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(live ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// d[16 x 8] += a[16 x 16] b[16 x 8], bf16 or f16 in, fp32 out
template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// two E4M3 codes (low byte first) -> two f16, exactly
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t pair) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)pair));
  return r;
}

template <int D_, bool FP8_>
struct Cfg {
  static constexpr int D = D_;
  static constexpr bool FP8 = FP8_;
  static constexpr int kRowBytes = FP8 ? D : 2 * D;
  static constexpr int kKeys = FP8 ? 32 : 16;          // keys of a warp in a tile
  static constexpr int kTile = kKeys * kWarps;         // keys of a unit
  static constexpr int kChunks = kRowBytes / 16;       // 16-byte chunks of a row
  static constexpr int kHalfBytes = kKeys * kRowBytes; // a warp's keys (or values) of a stage
  static constexpr int kStageBytes = 2 * kHalfBytes;   // = 16 * D * 4: a warp's output rows fit
  static constexpr int kStages = D == 128 ? 3 : 4;
  static constexpr int kSmem = kWarps * kStages * kStageBytes;
  static constexpr int kBlocks = D == 128 ? 2 : 3;     // resident blocks of an SM
  static_assert(kStageBytes >= kDecodeRows * D * 4, "merge area");
};

// where 16-byte chunk c of row r of a stage lies: rows of 128 or more bytes spread eight
// consecutive rows over the banks, 64-byte rows spread pairs of rows
template <int CH>
__device__ __forceinline__ uint32_t swz(int r, int c) {
  return (uint32_t)((r * CH + (c ^ (CH >= 8 ? (r & 7) : ((r >> 1) & 3)))) * 16);
}

// The tiles of a sequence's visible keys: the sinks first (if the window has left them behind),
// then the window.
struct Span {
  int len;    // kv_len, clamped to what the table can hold
  int sink;   // sink places before the window's first
  int lo;     // first place of the window
  int ts, n;  // sink tiles, all tiles (one at least)
};

template <int TILE>
__device__ __forceinline__ Span span_of(const AttnDims& a, int len) {
  Span s;
  s.len = min(max(len, 0), a.max_pages * a.page_size);
  s.lo = a.window ? max(0, s.len - a.window) : 0;
  s.sink = min(a.n_sink, s.lo);
  if (s.sink == s.lo) s.sink = s.lo = 0;  // no gap
  s.ts = (s.sink + TILE - 1) / TILE;
  s.n = max(1, s.ts + (s.len - s.lo + TILE - 1) / TILE);
  return s;
}

// A block's place in the row of units.
struct Cursor {
  int b, hr, tile;
  int64_t first;  // units before sequence b
  Span s;
};

template <int TILE>
__device__ __forceinline__ void advance(const DecodeParams& p, int hr_n, Cursor& c) {
  if (++c.tile < c.s.n) return;
  c.tile = 0;
  if (++c.hr < hr_n) return;
  c.hr = 0;
  c.first += (int64_t)c.s.n * hr_n;
  if (++c.b < p.a.B) c.s = span_of<TILE>(p.a, __ldg(p.kv_len + c.b));
}

template <class C>
__global__ void __launch_bounds__(kThreads, C::kBlocks) k_attn_decode(const DecodeParams p) {
  constexpr int D = C::D, TILE = C::kTile, CH = C::kChunks, NT = D / 8, KS = D / 16;
  constexpr bool FP8 = C::FP8;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float2 sml[kWarps][kDecodeRows];
  __shared__ int s_last;
  const AttnDims& a = p.a;
  const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31;
  const int g = lane >> 2, c4 = lane & 3;  // row and column group of an MMA fragment
  const int hr_n = a.Hkv * p.rt;
  pdl_wait_then_release();

  // ---- this block's run of units (each warp finds it alone) ----
  int64_t tiles = 0;
  for (int b = lane; b < a.B; b += 32) {
    const int len = __ldg(p.kv_len + b);
    if (warp == 0 && blockIdx.x == 0 && (len < 0 || len > a.max_pages * a.page_size))
      record_error(p.status, MOE_ERR_DEVICE_BOUNDS);
    tiles += span_of<TILE>(a, len).n;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) tiles += __shfl_xor_sync(0xffffffffu, tiles, o);
  const int64_t units = tiles * hr_n;
  const int64_t grid = min((int64_t)gridDim.x, units);
  if ((int64_t)blockIdx.x >= grid) return;
  const int64_t u0 = blockIdx.x * units / grid, u1 = (blockIdx.x + 1) * units / grid;

  Cursor cc;  // the unit to compute
  {
    int64_t before = 0;  // tiles before this round of 32 sequences
    for (int b0 = 0;; b0 += 32) {
      const int b = b0 + lane;
      const int mine = b < a.B ? span_of<TILE>(a, __ldg(p.kv_len + b)).n : 0;
      int64_t incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
      }
      const int64_t total = __shfl_sync(0xffffffffu, incl, 31);
      if (u0 < (before + total) * hr_n || b0 + 32 >= a.B) {
        const unsigned past = __ballot_sync(0xffffffffu, (before + incl) * hr_n <= u0);
        const int at = min(__popc(past), 31);
        cc.b = b0 + at;
        cc.first = (before + __shfl_sync(0xffffffffu, incl - mine, at)) * hr_n;
        break;
      }
      before += total;
    }
    cc.s = span_of<TILE>(a, __ldg(p.kv_len + cc.b));
    const int r = (int)(u0 - cc.first);
    cc.hr = r / cc.s.n;
    cc.tile = r - cc.hr * cc.s.n;
  }
  Cursor lc = cc;  // the unit to load

  uint8_t* ring = smem + warp * (C::kStages * C::kStageBytes);
  const uint32_t ring_u = smem_u32(ring);

  // the page of this lane's key of unit `c` (-1: not visible), and its row in the page
  const auto look_up = [&](const Cursor& c, int64_t u, int& page, int& row) {
    page = -1;
    row = 0;
    if (u >= u1 || lane >= C::kKeys) return;
    const bool in_sink = c.tile < c.s.ts;
    const int j = (in_sink ? c.tile * TILE : c.s.lo + (c.tile - c.s.ts) * TILE) +
                  warp * C::kKeys + lane;
    if (j >= (in_sink ? c.s.sink : c.s.len)) return;
    const int pg = (int)div_fast((uint32_t)j, a.page_div);
    row = j - pg * a.page_size;
    page = __ldg(p.block_table + (int64_t)c.b * a.max_pages + pg);
    if ((uint32_t)page >= (uint32_t)a.num_pages) {
      record_error(p.status, MOE_ERR_DEVICE_BOUNDS);
      page = -1;
    }
  };
  // copies this warp's keys and values of a unit into stage st
  const auto copy_in = [&](const Cursor& c, int page, int row, int st) {
    constexpr int RP = 32 / CH;  // rows of a pass
    const int64_t mine = page < 0 ? -1
                                  : (int64_t)page * a.page_stride + (int64_t)row * a.token_stride +
                                        (int64_t)(c.hr / p.rt) * a.head_stride;
    const int chunk = lane % CH;
    const uint32_t dst = ring_u + st * C::kStageBytes;
#pragma unroll
    for (int i = 0; i < C::kKeys / RP; ++i) {
      const int r = i * RP + lane / CH;
      const int64_t off = __shfl_sync(0xffffffffu, mine, r);
      const bool live = off >= 0;
      const int64_t at = live ? off * (FP8 ? 1 : 2) + chunk * 16 : 0;
      const uint32_t to = dst + swz<CH>(r, chunk);
      cp_async16(to, p.k_cache + at, live);
      cp_async16(to + C::kHalfBytes, p.v_cache + at, live);
    }
  };

  // ---- fill the ring ----
  int page, row;
  int64_t lu = u0;  // unit of the load cursor
  look_up(lc, lu, page, row);
#pragma unroll
  for (int st = 0; st < C::kStages; ++st) {
    if (lu < u1) {
      copy_in(lc, page, row, st);
      advance<TILE>(p, hr_n, lc);
      ++lu;
      look_up(lc, lu, page, row);
    }
    cp_async_commit();
  }

  uint32_t qf[KS][4];
  float acc[NT][4];
  float m[2], l[2];       // rows g and g + 8; m in the units of the raw scores
  float sc2[2] = {0, 0};  // raw score -> base-2 exponent
  bool fresh = true;

  int st = 0;
  for (int64_t u = u0; u < u1; ++u) {
    const int h = cc.hr / p.rt, row0 = (cc.hr - h * p.rt) * kDecodeRows;
    const int rows = min(kDecodeRows, a.G - row0);
    if (fresh) {  // a new item: its queries, and an empty softmax
      fresh = false;
      const uint16_t* qb =
          p.q + (int64_t)cc.b * a.qr_stride + (int64_t)(h * a.G + row0) * D;
      const float sc = a.scale * 1.4426950408889634f * (FP8 && p.k_scale ? __ldg(p.k_scale + h) : 1.f);
#pragma unroll
      for (int k = 0; k < KS; ++k) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {  // rows g, g+8, g, g+8; columns low, low, high, high
          const int qr = g + (r & 1) * 8;
          const int col = 16 * k + (FP8 ? 4 * c4 + (r >> 1) * 2 : 2 * c4 + (r >> 1) * 8);
          qf[k][r] = qr < rows ? *reinterpret_cast<const uint32_t*>(qb + (int64_t)qr * D + col) : 0u;
        }
      }
      sc2[0] = sc2[1] = sc;
      if (FP8) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float big = 0.f;
#pragma unroll
          for (int k = 0; k < KS; ++k) {
#pragma unroll
            for (int r = i; r < 4; r += 2)
              big = fmaxf(big, fmaxf(fabsf(bf16_lo(qf[k][r])), fabsf(bf16_hi(qf[k][r]))));
          }
          big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
          big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
          // 2^e with e = 14 - floor(log2 big), kept within the exponents of fp32
          const int e = min(100, max(-113, 141 - (int)(__float_as_uint(big) >> 23)));
          const float up = __uint_as_float((uint32_t)(127 + e) << 23);
          sc2[i] *= __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
          for (int k = 0; k < KS; ++k) {
#pragma unroll
            for (int r = i; r < 4; r += 2)
              qf[k][r] = pack_f16(bf16_lo(qf[k][r]) * up, bf16_hi(qf[k][r]) * up);
          }
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
      m[0] = m[1] = -INFINITY;
      l[0] = l[1] = 0.f;
    }

    cp_async_wait<C::kStages - 1>();
    __syncwarp();
    const uint32_t kb = ring_u + st * C::kStageBytes, vb = kb + C::kHalfBytes;
    const bool in_sink = cc.tile < cc.s.ts;
    // visible keys of this warp's part of the tile
    const int left = (in_sink ? cc.s.sink - cc.tile * TILE
                              : cc.s.len - cc.s.lo - (cc.tile - cc.s.ts) * TILE) -
                     warp * C::kKeys;
    if (left > 0) {
      // ---- scores: rows are query heads, columns this warp's keys ----
      constexpr int SN = C::kKeys / 8;
      float s[SN][4];
#pragma unroll
      for (int n = 0; n < SN; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
      if (!FP8) {
        // x4: keys 0-7 and 8-15, columns 16k..16k+7 and +8..+15
        const int r = (lane & 7) + ((lane >> 4) << 3), cc2 = (lane >> 3) & 1;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          uint32_t f[4];
          ldsm4(kb + swz<CH>(r, 2 * k + cc2), f);
          mma16816<false>(s[0], qf[k], f[0], f[1]);
          mma16816<false>(s[1], qf[k], f[2], f[3]);
        }
      } else {
        // x4: 8 keys each, 16 codes of a row: one k step of four key groups
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          uint32_t f[4];
          ldsm4(kb + swz<CH>(lane, k), f);
#pragma unroll
          for (int n = 0; n < 4; ++n)
            mma16816<true>(s[n], qf[k], e4m3x2_f16x2(f[n]), e4m3x2_f16x2(f[n] >> 16));
        }
      }
      if (left < C::kKeys) {
#pragma unroll
        for (int n = 0; n < SN; ++n) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (8 * n + 2 * c4 + (e & 1) >= left) s[n][e] = -INFINITY;
        }
      }
      // ---- running maximum and sum ----
      float mx[2] = {m[0], m[1]};
#pragma unroll
      for (int n = 0; n < SN; ++n) {
        mx[0] = fmaxf(mx[0], fmaxf(s[n][0], s[n][1]));
        mx[1] = fmaxf(mx[1], fmaxf(s[n][2], s[n][3]));
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
      }
      float base[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) base[i] = mx[i] == -INFINITY ? 0.f : mx[i] * sc2[i];
      if (__any_sync(0xffffffffu, mx[0] > m[0] || mx[1] > m[1])) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float f = m[i] == -INFINITY ? 0.f : ex2(fmaf(m[i], sc2[i], -base[i]));
          l[i] *= f;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            acc[n][2 * i] *= f;
            acc[n][2 * i + 1] *= f;
          }
          m[i] = mx[i];
        }
      }
      uint32_t pf[SN / 2][4], pl[SN / 2][4];
#pragma unroll
      for (int n = 0; n < SN; ++n) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float e0 = ex2(fmaf(s[n][2 * i], sc2[i], -base[i]));
          const float e1 = ex2(fmaf(s[n][2 * i + 1], sc2[i], -base[i]));
          l[i] += e0 + e1;
          const int at = (n & 1) * 2 + i;
          if (FP8) {
            pf[n >> 1][at] = pack_f16(e0, e1);
          } else {
            const uint32_t hi = pack_bf16(e0, e1);
            pf[n >> 1][at] = hi;
            pl[n >> 1][at] = pack_bf16(e0 - bf16_lo(hi), e1 - bf16_hi(hi));
          }
        }
      }
      // ---- o += p v ----
      if (!FP8) {
        const int r = lane & 15, hi = lane >> 4;
#pragma unroll
        for (int n = 0; n < NT / 2; ++n) {
          uint32_t f[4];  // keys 0-7, 8-15 of columns 16n..+7, then of the next eight
          ldsm4_t(vb + swz<CH>(r, 2 * n + hi), f);
          mma16816<false>(acc[2 * n], pf[0], f[0], f[1]);
          mma16816<false>(acc[2 * n + 1], pf[0], f[2], f[3]);
          mma16816<false>(acc[2 * n], pl[0], f[0], f[1]);
          mma16816<false>(acc[2 * n + 1], pl[0], f[2], f[3]);
        }
      } else {
#pragma unroll
        for (int n = 0; n < NT / 2; ++n) {
          uint32_t f[4];  // four groups of 8 keys, 16 columns in pairs
          ldsm4_t(vb + swz<CH>(lane, n), f);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            // keys 2c, 2c+1 (f[2k]) and 2c+8, 2c+9 (f[2k+1]); even columns, then odd ones
            mma16816<true>(acc[2 * n], pf[k], e4m3x2_f16x2(__byte_perm(f[2 * k], 0, 0x4420)),
                           e4m3x2_f16x2(__byte_perm(f[2 * k + 1], 0, 0x4420)));
            mma16816<true>(acc[2 * n + 1], pf[k], e4m3x2_f16x2(__byte_perm(f[2 * k], 0, 0x4431)),
                           e4m3x2_f16x2(__byte_perm(f[2 * k + 1], 0, 0x4431)));
          }
        }
      }
    }
    __syncwarp();

    // ---- the end of the item, or of this block's run: merge the warps ----
    const bool item_end = cc.tile + 1 == cc.s.n;
    if (item_end || u + 1 == u1) {
      fresh = true;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
        const float base = m[i] == -INFINITY ? -INFINITY : m[i] * sc2[i];
        if (c4 == 0) sml[warp][g + 8 * i] = make_float2(base, l[i]);
      }
      float* mine = reinterpret_cast<float*>(ring + st * C::kStageBytes);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = g + (e >> 1) * 8;
          // E4M3: tile pair n holds the even, then the odd columns of 16
          const int col = FP8 ? 16 * (n >> 1) + 4 * c4 + 2 * (e & 1) + (n & 1)
                              : 8 * n + 2 * c4 + (e & 1);
          mine[r * D + (col ^ ((r & 7) << 3))] = acc[n][e];
        }
      }
      __syncthreads();
      const int64_t item0 = cc.first + (int64_t)cc.hr * cc.s.n;  // the item's first unit
      const bool whole = item0 >= u0 && item_end;
      const int64_t c0 = ((item0 + 1) * grid - 1) / units;
      const int64_t c1 = ((item0 + cc.s.n) * grid - 1) / units;
      // a block has one item that began before it and one that it begins and does not end
      const int64_t slot = 2 * (int64_t)blockIdx.x + (item0 < u0 ? 0 : 1);
      const float vs = FP8 && p.v_scale ? __ldg(p.v_scale + h) : 1.f;
      const int64_t head0 = (int64_t)h * a.G + row0;
      for (int task = (int)threadIdx.x; task < rows * (D / 8); task += kThreads) {
        const int r = task / (D / 8), col = (task % (D / 8)) * 8;
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sml[w][r].x);
        float y[8] = {0, 0, 0, 0, 0, 0, 0, 0}, sum = 0.f;
        if (mm != -INFINITY) {
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float f = ex2(sml[w][r].x - mm);
            sum += f * sml[w][r].y;
            const float* src = reinterpret_cast<const float*>(
                smem + w * (C::kStages * C::kStageBytes) + st * C::kStageBytes);
            const float4* s4 =
                reinterpret_cast<const float4*>(src + r * D + (col ^ ((r & 7) << 3)));
            const float4 lo = s4[0], hi = s4[1];
            y[0] = fmaf(f, lo.x, y[0]); y[1] = fmaf(f, lo.y, y[1]);
            y[2] = fmaf(f, lo.z, y[2]); y[3] = fmaf(f, lo.w, y[3]);
            y[4] = fmaf(f, hi.x, y[4]); y[5] = fmaf(f, hi.y, y[5]);
            y[6] = fmaf(f, hi.z, y[6]); y[7] = fmaf(f, hi.w, y[7]);
          }
        }
        if (whole) {
          const float inv = sum > 0.f ? vs / sum : (sum == 0.f ? 0.f : sum);
          *reinterpret_cast<uint4*>(p.o + (int64_t)cc.b * a.o_stride + (head0 + r) * D + col) =
              make_uint4(pack_bf16(y[0] * inv, y[1] * inv), pack_bf16(y[2] * inv, y[3] * inv),
                         pack_bf16(y[4] * inv, y[5] * inv), pack_bf16(y[6] * inv, y[7] * inv));
          if (p.lse && col == 0)
            p.lse[(int64_t)cc.b * a.Hq + head0 + r] =
                sum == 0.f ? -INFINITY : mm * 0.6931471805599453f + logf(sum);
        } else {
          float4* dst = reinterpret_cast<float4*>(p.parts + (slot * kDecodeRows + r) * D + col);
          __stcg(dst, make_float4(y[0], y[1], y[2], y[3]));
          __stcg(dst + 1, make_float4(y[4], y[5], y[6], y[7]));
          if (col == 0) __stcg(p.ml + slot * kDecodeRows + r, make_float2(mm, sum));
        }
      }
      if (!whole) {
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) {
          const int old = atomicAdd(p.counters + c0, 1);
          s_last = old == (int)(c1 - c0);
          if (s_last) p.counters[c0] = 0;  // left as it was found
        }
        __syncthreads();
        if (s_last) {
          __threadfence();
          for (int task = (int)threadIdx.x; task < rows * (D / 8); task += kThreads) {
            const int r = task / (D / 8), col = (task % (D / 8)) * 8;
            float mm = -INFINITY, sum = 0.f, y[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            for (int64_t c = c0; c <= c1; ++c) {
              const int64_t sl = 2 * c + (c == c0 ? 1 : 0);
              mm = fmaxf(mm, __ldcg(p.ml + sl * kDecodeRows + r).x);
            }
            if (mm != -INFINITY) {
              for (int64_t c = c0; c <= c1; ++c) {
                const int64_t sl = 2 * c + (c == c0 ? 1 : 0);
                const float2 v = __ldcg(p.ml + sl * kDecodeRows + r);
                const float f = ex2(v.x - mm);
                sum += f * v.y;
                const float4* src =
                    reinterpret_cast<const float4*>(p.parts + (sl * kDecodeRows + r) * D + col);
                const float4 lo = __ldcg(src), hi = __ldcg(src + 1);
                y[0] = fmaf(f, lo.x, y[0]); y[1] = fmaf(f, lo.y, y[1]);
                y[2] = fmaf(f, lo.z, y[2]); y[3] = fmaf(f, lo.w, y[3]);
                y[4] = fmaf(f, hi.x, y[4]); y[5] = fmaf(f, hi.y, y[5]);
                y[6] = fmaf(f, hi.z, y[6]); y[7] = fmaf(f, hi.w, y[7]);
              }
            }
            const float inv = sum > 0.f ? vs / sum : (sum == 0.f ? 0.f : sum);
            *reinterpret_cast<uint4*>(p.o + (int64_t)cc.b * a.o_stride + (head0 + r) * D + col) =
                make_uint4(pack_bf16(y[0] * inv, y[1] * inv), pack_bf16(y[2] * inv, y[3] * inv),
                           pack_bf16(y[4] * inv, y[5] * inv), pack_bf16(y[6] * inv, y[7] * inv));
            if (p.lse && col == 0)
              p.lse[(int64_t)cc.b * a.Hq + head0 + r] =
                  sum == 0.f ? -INFINITY : mm * 0.6931471805599453f + logf(sum);
          }
        }
      }
      __syncthreads();  // the merge area is a stage: read before it is filled again
    }

    // ---- the next unit to load, into the stage just consumed ----
    if (lu < u1) {
      copy_in(lc, page, row, st);
      advance<TILE>(p, hr_n, lc);
      ++lu;
      look_up(lc, lu, page, row);
    }
    cp_async_commit();
    if (++st == C::kStages) st = 0;
    advance<TILE>(p, hr_n, cc);
  }
  cp_async_wait<0>();
}

template <class C>
cudaError_t launch(const DecodeParams& p, cudaStream_t st) {
  auto kern = k_attn_decode<C>;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  count_launches(1);
  const int grid = num_sms() * C::kBlocks;
  return launch_pdl(kern, dim3((unsigned)(grid < kAttnMaxCtas ? grid : kAttnMaxCtas)),
                    dim3(kThreads), C::kSmem, st, p);
}

}  // namespace

cudaError_t launch_attn_decode(const AttnDims& a, const void* q, const void* k_cache,
                               const void* v_cache, const float* k_scale, const float* v_scale,
                               const int32_t* block_table, const int32_t* kv_len, void* o,
                               float* lse, char* ws, const AttnWs& L, cudaStream_t st) {
  DecodeParams p{};
  p.a = a;
  p.q = static_cast<const uint16_t*>(q);
  p.k_cache = static_cast<const uint8_t*>(k_cache);
  p.v_cache = static_cast<const uint8_t*>(v_cache);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.block_table = block_table;
  p.kv_len = kv_len;
  p.o = static_cast<uint16_t*>(o);
  p.lse = lse;
  p.status = reinterpret_cast<int*>(ws + L.status);
  p.counters = reinterpret_cast<int*>(ws + L.counters);
  p.parts = reinterpret_cast<float*>(ws + L.parts);
  p.ml = reinterpret_cast<float2*>(ws + L.ml);
  p.rt = (a.G + kDecodeRows - 1) / kDecodeRows;
  if (a.D == 64)
    return a.fp8 ? launch<Cfg<64, true>>(p, st) : launch<Cfg<64, false>>(p, st);
  return a.fp8 ? launch<Cfg<128, true>>(p, st) : launch<Cfg<128, false>>(p, st);
}

}  // namespace moe
