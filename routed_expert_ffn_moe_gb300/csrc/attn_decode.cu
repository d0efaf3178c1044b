// Attention of one new token per sequence over the paged cache.
//
//   s_j = scale q.k_j over the visible places j,  o = sum_j e^(s_j - m) v_j / l,
//   m = max_j s_j,  l = sum_j e^(s_j - m),  lse = m + ln l
//
// What bounds it: HBM. Every visible key and value is read once for each 16 query heads of its key
// head, 2 G multiply-adds an element, far below the tensor cores' rate even padded to 16 query heads.
//
// Work split. An item is one sequence, one key head and up to 16 of its query heads; a unit is
// one tile of an item's visible keys (64 of 256 bytes, in general 32 KB of keys and values), or the
// end of an item, which costs about as much as a tile. All units of the batch in a row are cut
// into equal runs, one per block of a grid that fills the SMs, whatever the lengths are: a
// block ends one item, does some whole ones and begins another. An item that spans blocks leaves
// one partial (m, l, unnormalised o) per block; a second kernel (k_attn_join), whose blocks share
// an item's rows and columns between them and its parts between lanes, joins them in a fixed
// order, so the result does not depend on timing.
//
// Inside a block every warp has its own quarter of the keys of each tile and its own ring of
// cp.async stages: it fetches the page of each key, copies the rows (zeros for places that are
// not visible: what the cache holds there never enters a product), and runs the running softmax
// on m16n8k16 MMAs, the 16 rows being query heads. Nothing synchronises the warps until an
// item ends, when they merge through the stage that was just consumed.
//
// Probabilities of a bf16 cache enter the product with v as two bf16 terms (2^-16 relative): the
// tensor cores have room, and one term alone would be the largest error of the result. Those of an
// E4M3 cache are one f16 term (2^-11 relative down to 2^-28 of the largest, 2^-39 of that below):
// its codes carry 2^-4 themselves.
//
// E4M3 codes enter the MMAs as f16 (exactly). The queries become f16 too, each row times the
// power of two that brings its largest element to [2^14, 2^15), taken back in the scores'
// scale: elements above 2^-28 of the row's largest are exact. An 8-bit row is read in 16-bit
// pairs, which permutes the contraction index of q.k (the queries are loaded in the same order)
// and the columns of v (stored back in place).
//
// Measured, of a copy rate of 6772 GB/s, 8 key heads of 128, 64 query heads: 256 sequences of 2048
// to 8192 places, bf16, 812 us, 0.98; one of 131071, 89 us, 0.89, of 524288, 324 us, 0.98; 64 sequences
// of 2048 places in E4M3 pages of 16, 63 us, 0.63, of 32768, 769 us, 0.83, in pages of 64, 701 us, 0.91
// (runs of 2 KB, the conversions, and the 8 warps that the registers leave an SM); one of 1003 places, 7.1
// us: the start of two kernels. Wider groups read again: 64 sequences of 8192 places, one key head of
// 128, bf16, 16, 32, 64, 128 query heads: 56, 93, 172, 264 us.
#include "attn.h"
#include "sm100_ptx.cuh"

namespace moe {
namespace {

using namespace ptx;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
// The maximum that a warp or a part publishes where no score was above -inf. Finite, so that its factor
// is 0 or 1 and never a NaN: whether a row saw anything is told by its sum, which is a NaN where a
// score was (no maximum holds a NaN).
constexpr float kNoMax = -3e38f;

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
  float* parts;
  float2* ml;
  int rt;      // items of a key head: ceil(G / 16)
  int blocks;  // of the grid
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

// The loads and products below are not volatile, so that the compiler may interleave the loads of
// later fragments with earlier products. What keeps a load between the arrival of its stage and
// the stage's next copy are its address, which passes through `after_wait`, and its results, which
// pass through `before_refill`.
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(addr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(addr));
}
__device__ __forceinline__ void after_wait(uint32_t& addr) { asm volatile("" : "+r"(addr) : : "memory"); }
template <int N>
__device__ __forceinline__ void before_refill(float (&acc)[N][4]) {
#pragma unroll
  for (int n = 0; n < N; ++n)
    asm volatile("" : "+f"(acc[n][0]), "+f"(acc[n][1]), "+f"(acc[n][2]), "+f"(acc[n][3]) : : "memory");
}

// d[16 x 8] += a[16 x 16] b[16 x 8], bf16 or f16 in, fp32 out
template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
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
  // Exponents are formed this much higher where probabilities are f16: the largest becomes 2^14, and
  // what is below 2^-39 of it, not 2^-25, is lost (of one key; a block may hold 10^5 of them).
  static constexpr float kUp = FP8 ? 14.f : 0.f;
  static constexpr int kRowBytes = FP8 ? D : 2 * D;
  static constexpr int kKeys = 4096 / kRowBytes;       // keys of a warp in a tile: 8 KB with values
  static constexpr int kTile = kKeys * kWarps;         // keys of a unit
  static constexpr int kChunks = kRowBytes / 16;       // 16-byte chunks of a row
  static constexpr int kHalfBytes = kKeys * kRowBytes; // a warp's keys (or values) of a stage
  static constexpr int kStageBytes = 2 * kHalfBytes;   // a warp's output rows fit for the merge
  static constexpr int kLook = kKeys > 32 ? kKeys / 32 : 1;  // keys that a lane looks up
  // Resident blocks of an SM, which share its registers and shared memory: three of two stages
  // where a warp's fragments fit in 168 registers and the conversions of E4M3 keep it busier than
  // the loads, else two of three. 96 sequences of 2 key heads of 64, E4M3, three against two, us:
  // 32768 places 149 against 165, 8192 47 against 50, 1024 13.7 against 13.6; bf16, 247 against
  // 254, 70 against 72, 18.5 against 18.0. 64 sequences of 8 key heads of 128, E4M3: 710 against
  // 769, 199 against 206, but 68 against 63 at 2048 (they spill, and items end more often).
  static constexpr int kBlocks = FP8 && D == 64 ? 3 : 2;
  static constexpr int kStages = kBlocks == 3 ? 2 : 3;
  static constexpr int kSmem = kWarps * kStages * kStageBytes;
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
  int ts, n;  // sink tiles, all tiles (one at least); the item has n + 1 units
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

// A block's place in the row of units; unit n of an item is its end.
struct Cursor {
  int b, hr, tile;
  int64_t first;  // units before sequence b
  Span s;
};

// To the next tile; returns the units passed: two past the end of an item.
template <int TILE>
__device__ __forceinline__ int advance(const DecodeParams& p, int hr_n, Cursor& c) {
  if (++c.tile < c.s.n) return 1;
  c.tile = 0;
  if (++c.hr < hr_n) return 2;
  c.hr = 0;
  c.first += (int64_t)(c.s.n + 1) * hr_n;
  if (++c.b >= p.a.B) return 2;
  const int len = __ldg(p.kv_len + c.b);
  if (len < 0 || len > p.a.max_pages * p.a.page_size)
    record_error(p.status, MOE_ERR_DEVICE_BOUNDS);
  c.s = span_of<TILE>(p.a, len);
  return 2;
}

// n / d of non-negative numbers: a 32-bit division where both fit
__device__ __forceinline__ int64_t div_s(int64_t n, int64_t d) {
  return ((n | d) >> 32) == 0 ? (int64_t)((uint32_t)n / (uint32_t)d) : n / d;
}

// Lengths of the batch, in one warp: lane i holds those of sequences i, i + 32, ..., of the first
// 32 * kHeld in registers, so that one round of loads serves the sum and the search.
template <int TILE>
struct Units {
  static constexpr int kHeld = 8;
  int held[kHeld];
  int64_t n;     // all units
  int grid;      // blocks that take some
  int64_t each;  // units of a block; the first `more` blocks take one more
  int more;

  __device__ __forceinline__ int units_of(const DecodeParams& p, int len) const {
    return span_of<TILE>(p.a, len).n + 1;
  }

  __device__ __forceinline__ void count(const DecodeParams& p) {
    const int lane = (int)threadIdx.x & 31, B = p.a.B;
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      held[i] = lane + 32 * i < B ? __ldcg(p.kv_len + lane + 32 * i) : 0;
    int64_t sum = 0;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) sum += lane + 32 * i < B ? units_of(p, held[i]) : 0;
    for (int b = lane + 32 * kHeld; b < B; b += 32) sum += units_of(p, __ldcg(p.kv_len + b));
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    n = sum * p.a.Hkv * p.rt;
    grid = (int)min((int64_t)p.blocks, n);
    each = div_s(n, grid);
    more = (int)(n - each * grid);
  }

  // the first unit of block c
  __device__ __forceinline__ int64_t start(int c) const { return c * each + min(c, more); }
  // the block that takes unit u
  __device__ __forceinline__ int block_of(int64_t u) const {
    const int64_t longer = more * (each + 1);  // units of the blocks that take one more
    return (int)(u < longer ? div_s(u, each + 1) : more + div_s(u - longer, each));
  }

  __device__ __forceinline__ Cursor find(const DecodeParams& p, int64_t u) const {
    const int lane = (int)threadIdx.x & 31, B = p.a.B, hr_n = p.a.Hkv * p.rt;
    Cursor c;
    int64_t before = 0;  // units of a head before this round of 32 sequences
    int len = 0;
    for (int b0 = 0;; b0 += 32) {
      int mine = 0;
#pragma unroll
      for (int i = 0; i < kHeld; ++i) mine = b0 == 32 * i ? held[i] : mine;
      if (b0 >= 32 * kHeld && b0 + lane < B) mine = __ldcg(p.kv_len + b0 + lane);
      const int64_t some = b0 + lane < B ? units_of(p, mine) : 0;
      int64_t incl = some;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
      }
      const int64_t total = __shfl_sync(0xffffffffu, incl, 31);
      if (u < (before + total) * hr_n || b0 + 32 >= B) {
        const unsigned past = __ballot_sync(0xffffffffu, (before + incl) * hr_n <= u);
        const int at = min(__popc(past), 31);
        c.b = b0 + at;
        c.first = (before + __shfl_sync(0xffffffffu, incl - some, at)) * hr_n;
        len = __shfl_sync(0xffffffffu, mine, at);
        break;
      }
      before += total;
    }
    if (len < 0 || len > p.a.max_pages * p.a.page_size)
      record_error(p.status, MOE_ERR_DEVICE_BOUNDS);
    c.s = span_of<TILE>(p.a, len);
    const int r = (int)(u - c.first);
    c.hr = r / (c.s.n + 1);
    c.tile = r - c.hr * (c.s.n + 1);
    return c;
  }
};

template <class C>
__global__ void __launch_bounds__(kThreads, C::kBlocks) k_attn_decode(const DecodeParams p) {
  constexpr int D = C::D, TILE = C::kTile, CH = C::kChunks, NT = D / 8, KS = D / 16;
  constexpr bool FP8 = C::FP8;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float2 sml[kWarps][kDecodeRows];
  const AttnDims& a = p.a;
  const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31;
  const int g = lane >> 2, c4 = lane & 3;  // row and column group of an MMA fragment
  const int hr_n = a.Hkv * p.rt;
  pdl_wait_then_release();

  // this block's run of units (each warp finds it alone)
  Units<TILE> un;
  un.count(p);
  if ((int)blockIdx.x >= un.grid) return;
  const int64_t u0 = un.start((int)blockIdx.x), u1 = un.start((int)blockIdx.x + 1);
  Cursor cc = un.find(p, u0);  // the unit to compute
  int64_t cu = u0;             // its number
  if (cc.tile == cc.s.n) {     // the run begins with an item's end
    cc.tile = cc.s.n - 1;
    cu += advance<TILE>(p, hr_n, cc) - 1;
  }
  Cursor lc = cc;  // the unit to load

  uint8_t* ring = smem + warp * (C::kStages * C::kStageBytes);
  const uint32_t ring_u = smem_u32(ring);

  // the pages of this lane's keys (lane, lane + 32) of unit `c`, and their rows (-1: not visible);
  // nothing here waits for a page
  const auto look_up = [&](const Cursor& c, int64_t u, int (&page)[C::kLook], int (&row)[C::kLook]) {
#pragma unroll
    for (int i = 0; i < C::kLook; ++i) {
      page[i] = 0;
      row[i] = -1;
      const int key = 32 * i + lane;
      if (u >= u1 || key >= C::kKeys) continue;
      const bool in_sink = c.tile < c.s.ts;
      const int j = (in_sink ? c.tile * TILE : c.s.lo + (c.tile - c.s.ts) * TILE) +
                    warp * C::kKeys + key;
      if (j >= (in_sink ? c.s.sink : c.s.len)) continue;
      const int pg = (int)div_fast((uint32_t)j, a.page_div);
      row[i] = j - pg * a.page_size;
      page[i] = __ldg(p.block_table + (int64_t)c.b * a.max_pages + pg);
    }
  };
  // copies this warp's keys and values of a unit into stage st
  const auto copy_in = [&](const Cursor& c, const int (&page)[C::kLook],
                           const int (&row)[C::kLook], int st) {
    constexpr int RP = 32 / CH;  // rows of a pass
    int64_t mine[C::kLook];
#pragma unroll
    for (int i = 0; i < C::kLook; ++i) {
      const bool there = (uint32_t)page[i] < (uint32_t)a.num_pages;
      if (row[i] >= 0 && !there) record_error(p.status, MOE_ERR_DEVICE_BOUNDS);
      mine[i] = row[i] < 0 || !there ? -1
                                     : (int64_t)page[i] * a.page_stride +
                                           (int64_t)row[i] * a.token_stride +
                                           (int64_t)(c.hr / p.rt) * a.head_stride;
    }
    const int chunk = lane % CH;
    const uint32_t dst = ring_u + st * C::kStageBytes;
#pragma unroll
    for (int i = 0; i < C::kKeys / RP; ++i) {
      const int r = i * RP + lane / CH;
      const int64_t off = __shfl_sync(0xffffffffu, mine[i * RP / 32], r & 31);
      const bool live = off >= 0;
      const int64_t at = live ? off * (FP8 ? 1 : 2) + chunk * 16 : 0;
      const uint32_t to = dst + swz<CH>(r, chunk);
      cp_async16(to, p.k_cache + at, live);
      cp_async16(to + C::kHalfBytes, p.v_cache + at, live);
    }
  };

  uint32_t qf[KS][4];
  float acc[NT][4];
  float m[2], l[2];       // rows g and g + 8; m in the units of the raw scores
  float sc2[2] = {0, 0};  // raw score -> base-2 exponent
  // the queries of an item, as they lie; an item's are asked for before the one before is merged
  const auto load_q = [&](const Cursor& c) {
    const int h = c.hr / p.rt, row0 = (c.hr - h * p.rt) * kDecodeRows;
    const int rows = min(kDecodeRows, a.G - row0);
    const uint16_t* qb = p.q + (int64_t)c.b * a.qr_stride + (int64_t)(h * a.G + row0) * D;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {  // rows g, g+8, g, g+8; columns low, low, high, high
        const int qr = g + (r & 1) * 8;
        const int col = 16 * k + (FP8 ? 4 * c4 + (r >> 1) * 2 : 2 * c4 + (r >> 1) * 8);
        qf[k][r] = qr < rows ? *reinterpret_cast<const uint32_t*>(qb + (int64_t)qr * D + col) : 0u;
      }
    }
  };
  bool fresh = true;
  if (cu < u1) load_q(cc);

  // ---- fill the ring: all look-ups first, so that their latencies pass together ----
  int page[C::kLook], row[C::kLook];
  int64_t lu = cu;  // unit of the load cursor
  {
    Cursor at[C::kStages];
    int pages[C::kStages][C::kLook], rows_of[C::kStages][C::kLook];
    bool is[C::kStages];
#pragma unroll
    for (int st = 0; st < C::kStages; ++st) {
      is[st] = lu < u1;
      if (is[st]) {
        at[st] = lc;
        look_up(lc, lu, pages[st], rows_of[st]);
        lu += advance<TILE>(p, hr_n, lc);
      }
    }
    look_up(lc, lu, page, row);
#pragma unroll
    for (int st = 0; st < C::kStages; ++st) {
      if (is[st]) copy_in(at[st], pages[st], rows_of[st], st);
      cp_async_commit();
    }
  }

  int st = 0;
  while (cu < u1) {
    const int h = cc.hr / p.rt, row0 = (cc.hr - h * p.rt) * kDecodeRows;
    const int rows = min(kDecodeRows, a.G - row0);
    if (fresh) {  // a new item: an empty softmax, and the queries in f16 for E4M3
      fresh = false;
      sc2[0] = sc2[1] =
          a.scale * 1.4426950408889634f * (FP8 && p.k_scale ? __ldg(p.k_scale + h) : 1.f);
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
    uint32_t kb = ring_u + st * C::kStageBytes;
    after_wait(kb);
    const uint32_t vb = kb + C::kHalfBytes;
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
#pragma unroll
          for (int n = 0; n < SN; n += 2) {
            uint32_t f[4];
            ldsm4(kb + swz<CH>(8 * n + r, 2 * k + cc2), f);
            mma16816<false>(s[n], qf[k], f[0], f[1]);
            mma16816<false>(s[n + 1], qf[k], f[2], f[3]);
          }
        }
      } else {
        // x4: 8 keys each, 16 codes of a row: one k step of four key groups
#pragma unroll
        for (int k = 0; k < KS; ++k) {
#pragma unroll
          for (int n = 0; n < SN; n += 4) {
            uint32_t f[4];
            ldsm4(kb + swz<CH>(8 * n + lane, k), f);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              mma16816<true>(s[n + e], qf[k], e4m3x2_f16x2(f[e]), e4m3x2_f16x2(f[e] >> 16));
          }
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
      float top[2], base[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        top[i] = mx[i] == -INFINITY ? 0.f : mx[i] * sc2[i];
        base[i] = top[i] - C::kUp;
      }
      if (__any_sync(0xffffffffu, mx[0] > m[0] || mx[1] > m[1])) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float f = m[i] == -INFINITY ? 0.f : ex2(fmaf(m[i], sc2[i], -top[i]));
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
#pragma unroll
          for (int k = 0; k < SN / 2; ++k) {
            uint32_t f[4];  // 16 keys: 0-7, 8-15 of columns 16n..+7, then of the next eight
            ldsm4_t(vb + swz<CH>(16 * k + r, 2 * n + hi), f);
            mma16816<false>(acc[2 * n], pf[k], f[0], f[1]);
            mma16816<false>(acc[2 * n + 1], pf[k], f[2], f[3]);
            mma16816<false>(acc[2 * n], pl[k], f[0], f[1]);
            mma16816<false>(acc[2 * n + 1], pl[k], f[2], f[3]);
          }
        }
      } else {
#pragma unroll
        for (int n = 0; n < NT / 2; ++n) {
#pragma unroll
          for (int k0 = 0; k0 < SN / 2; k0 += 2) {
            uint32_t f[4];  // four groups of 8 keys, 16 columns in pairs
            ldsm4_t(vb + swz<CH>(16 * k0 + lane, n), f);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              // keys 2c, 2c+1 (f[2k]) and 2c+8, 2c+9 (f[2k+1]); even columns, then odd ones
              mma16816<true>(acc[2 * n], pf[k0 + k],
                             e4m3x2_f16x2(__byte_perm(f[2 * k], 0, 0x4420)),
                             e4m3x2_f16x2(__byte_perm(f[2 * k + 1], 0, 0x4420)));
              mma16816<true>(acc[2 * n + 1], pf[k0 + k],
                             e4m3x2_f16x2(__byte_perm(f[2 * k], 0, 0x4431)),
                             e4m3x2_f16x2(__byte_perm(f[2 * k + 1], 0, 0x4431)));
            }
          }
        }
      }
    }
    before_refill(acc);
    __syncwarp();

    // ---- the end of the item, or of this block's run: merge the warps ----
    const bool item_end = cc.tile + 1 == cc.s.n;
    Cursor nc = cc;
    const int64_t nu = cu + advance<TILE>(p, hr_n, nc);
    if (item_end || nu >= u1) {
      fresh = true;
      if (nu < u1) load_q(nc);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
        const float base = m[i] == -INFINITY ? kNoMax : m[i] * sc2[i] - C::kUp;
        if (c4 == 0) sml[warp][g + 8 * i] = make_float2(base, l[i]);
      }
      float* mine = reinterpret_cast<float*>(ring + st * C::kStageBytes);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float* to = mine + (g + 8 * i) * D;
        const int x = (g & 7) << 3;
        if (FP8) {  // tile pair n holds the even, then the odd columns of 16
#pragma unroll
          for (int n = 0; n < NT; n += 2)
            *reinterpret_cast<float4*>(to + ((8 * n + 4 * c4) ^ x)) =
                make_float4(acc[n][2 * i], acc[n + 1][2 * i], acc[n][2 * i + 1],
                            acc[n + 1][2 * i + 1]);
        } else {
#pragma unroll
          for (int n = 0; n < NT; ++n)
            *reinterpret_cast<float2*>(to + ((8 * n + 2 * c4) ^ x)) =
                make_float2(acc[n][2 * i], acc[n][2 * i + 1]);
        }
      }
      __syncthreads();
      const int64_t item0 = cc.first + (int64_t)cc.hr * (cc.s.n + 1);  // the item's first unit
      const bool whole = item0 >= u0 && item_end;
      // a block has one item that began before it and one that it begins and does not end
      const int64_t slot = 2 * (int64_t)blockIdx.x + (item0 < u0 ? 0 : 1);
      const float vs = FP8 && p.v_scale ? __ldg(p.v_scale + h) : 1.f;
      const int64_t head0 = (int64_t)h * a.G + row0;
      for (int task = (int)threadIdx.x; task < rows * (D / 8); task += kThreads) {
        const int r = task / (D / 8), col = (task % (D / 8)) * 8;
        float mm = kNoMax;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sml[w][r].x);
        float y[8] = {0, 0, 0, 0, 0, 0, 0, 0}, sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float f = ex2(sml[w][r].x - mm);
          sum += f * sml[w][r].y;
          const float* src = reinterpret_cast<const float*>(
              smem + w * (C::kStages * C::kStageBytes) + st * C::kStageBytes);
          const float4* s4 = reinterpret_cast<const float4*>(src + r * D + (col ^ ((r & 7) << 3)));
          const float4 lo = s4[0], hi = s4[1];
          y[0] = fmaf(f, lo.x, y[0]); y[1] = fmaf(f, lo.y, y[1]);
          y[2] = fmaf(f, lo.z, y[2]); y[3] = fmaf(f, lo.w, y[3]);
          y[4] = fmaf(f, hi.x, y[4]); y[5] = fmaf(f, hi.y, y[5]);
          y[6] = fmaf(f, hi.z, y[6]); y[7] = fmaf(f, hi.w, y[7]);
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
      __syncthreads();  // the merge area is a stage: read before it is filled again
    }

    // ---- the next unit to load, into the stage just consumed ----
    if (lu < u1) {
      copy_in(lc, page, row, st);
      lu += advance<TILE>(p, hr_n, lc);
      look_up(lc, lu, page, row);
    }
    cp_async_commit();
    if (++st == C::kStages) st = 0;
    cc = nc;
    cu = nu;
  }
  cp_async_wait<0>();
}

// Joins the parts of the items that span blocks. Block c - 1 looks at the boundary between blocks c - 1
// and c of k_attn_decode: if it lies inside an item, the blocks of that item's boundaries share its
// (row, eight columns) tasks; the lanes of a group take a task's parts in turn, each with a running
// maximum, and meet in a butterfly. Blocks with nothing to join wait for k_attn_decode too: the kernel
// after this one waits for this one alone. Bound by latency: its blocks find their boundary while
// k_attn_decode runs, and joining in k_attn_decode instead (the last block to arrive joins an item) took
// 9.5 us against 7.5 for one sequence of 1003 places, and with one key head over 131072 places, whose
// parts then all fall to one block, 211 against 27.
template <class C>
__global__ void __launch_bounds__(kThreads) k_attn_join(const DecodeParams p) {
  constexpr int D = C::D;
  const AttnDims& a = p.a;
  // the lengths were there before k_attn_decode began
  Units<C::kTile> un;
  un.count(p);
  const int c = (int)blockIdx.x + 1;
  Cursor cur;
  bool inside = c < un.grid;
  if (inside) {
    cur = un.find(p, un.start(c));
    inside = cur.tile != 0 && cur.tile != cur.s.n;  // else between two items
  }
  if (!inside) {
    pdl_wait_then_release();
    return;
  }
  const int64_t item0 = cur.first + (int64_t)cur.hr * (cur.s.n + 1);
  const int c0 = un.block_of(item0), c1 = un.block_of(item0 + cur.s.n - 1);
  const int h = cur.hr / p.rt, row0 = (cur.hr - h * p.rt) * kDecodeRows;
  const int rows = min(kDecodeRows, a.G - row0), tasks = rows * (D / 8);
  const int t0 = (c - c0 - 1) * tasks / (c1 - c0), t1 = (c - c0) * tasks / (c1 - c0);
  int lanes = 2;  // of a task
  while (lanes < 32 && lanes < c1 - c0 + 1) lanes *= 2;
  const int mine = (int)threadIdx.x % lanes;
  const float vs = C::FP8 && p.v_scale ? __ldg(p.v_scale + h) : 1.f;
  pdl_wait_then_release();
  const int per = kThreads / lanes;
  for (int first = t0; first < t1; first += per) {
    const int task = first + (int)threadIdx.x / lanes;
    const bool live = task < t1;
    const int r = live ? task / (D / 8) : 0, col = live ? (task % (D / 8)) * 8 : 0;
    float m = kNoMax, sum = 0.f, y[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int part = c0 + mine; live && part <= c1; part += lanes) {
      // the part that began the item is its block's second, the others are their blocks' first
      const int64_t at = (int64_t)(2 * part + (part == c0 ? 1 : 0)) * kDecodeRows + r;
      const float2 ml = __ldcg(p.ml + at);
      const float4* src = reinterpret_cast<const float4*>(p.parts + at * D + col);
      const float4 lo = __ldcg(src), hi = __ldcg(src + 1);
      const float to = fmaxf(m, ml.x), f = ex2(m - to), g = ex2(ml.x - to);
      const float z[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
      sum = sum * f + ml.y * g;
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = fmaf(z[e], g, y[e] * f);
      m = to;
    }
    float all = m;
    for (int o = lanes / 2; o; o >>= 1) all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, o));
    const float f = ex2(m - all);
    sum *= f;
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] *= f;
    for (int o = lanes / 2; o; o >>= 1) {
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] += __shfl_xor_sync(0xffffffffu, y[e], o);
    }
    if (live && mine == 0) {
      const float inv = sum == 0.f ? 0.f : vs / sum;
      const int64_t head = (int64_t)h * a.G + row0 + r;
      *reinterpret_cast<uint4*>(p.o + (int64_t)cur.b * a.o_stride + head * D + col) =
          make_uint4(pack_bf16(y[0] * inv, y[1] * inv), pack_bf16(y[2] * inv, y[3] * inv),
                     pack_bf16(y[4] * inv, y[5] * inv), pack_bf16(y[6] * inv, y[7] * inv));
      if (p.lse && col == 0)
        p.lse[(int64_t)cur.b * a.Hq + head] =
            sum == 0.f ? -INFINITY : all * 0.6931471805599453f + logf(sum);
    }
  }
}

// the most units that a batch of this shape can have
int64_t most_units(const DecodeParams& p, int tile) {
  const int64_t places = (int64_t)p.a.max_pages * p.a.page_size;
  const int64_t seen = p.a.window ? (int64_t)p.a.window + p.a.n_sink : places;
  const int64_t tiles =  // two ragged ends, and the unit that ends the item
      ((seen < places ? seen : places) + tile - 1) / tile + 2;
  return tiles * p.a.B * p.a.Hkv * p.rt;
}

template <class C>
cudaError_t launch(DecodeParams& p, cudaStream_t st) {
  auto kern = k_attn_decode<C>;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  // a block for every place on the SMs, but no more than there can be units
  const int64_t most = most_units(p, C::kTile);
  p.blocks = num_sms() * C::kBlocks;
  if (p.blocks > kAttnMaxCtas) p.blocks = kAttnMaxCtas;
  if (p.blocks > most) p.blocks = (int)most;
  count_launches(p.blocks > 1 ? 2 : 1);
  e = launch_pdl(kern, dim3((unsigned)p.blocks), dim3(kThreads), C::kSmem, st, p);
  if (e != cudaSuccess || p.blocks == 1) return e;
  return launch_pdl(k_attn_join<C>, dim3((unsigned)p.blocks - 1), dim3(kThreads), 0, st, p);
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
  p.parts = reinterpret_cast<float*>(ws + L.parts);
  p.ml = reinterpret_cast<float2*>(ws + L.ml);
  p.rt = (a.G + kDecodeRows - 1) / kDecodeRows;
  if (a.D == 64)
    return a.fp8 ? launch<Cfg<64, true>>(p, st) : launch<Cfg<64, false>>(p, st);
  return a.fp8 ? launch<Cfg<128, true>>(p, st) : launch<Cfg<128, false>>(p, st);
}

}  // namespace moe
