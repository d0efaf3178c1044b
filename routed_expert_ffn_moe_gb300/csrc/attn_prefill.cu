// Attention of any number of new tokens per sequence over the paged cache (prompts, and chunks of
// prompts), on tcgen05 tensor cores.
//
//   s_ij = scale q_i.k_j over the places j that token i sees, o_i = sum_j softmax(s_i)_j v_j
//
// What bounds it: the tensor cores, 4 D flops per visible (query head, key) pair; next to them
// the exponentials, one per pair.
//
// Tiles. The G query heads of a key head share its keys, so a tile of 128 rows is 128/G
// consecutive tokens times G heads (row t*G + g; when G does not divide 128 the last rows are
// idle), and the key axis runs in tiles of 128 places. A block holds two such row tiles of one
// sequence and key head and walks the key tiles that any of their rows sees: the sinks, then from
// the window's first place to the last token. While the softmax works on one row tile's
// scores the tensor cores work on the other's.
//
// Tensor memory: per row tile 128 columns of scores S (fp32) and D columns of output O (fp32).
// The probabilities P (bf16) overwrite S and are the A operand of the second product from there;
// K is K-major and V MN-major as TMA lays both down (rows of places, 128-byte swizzle).
//
// Warps: 0-3 softmax of row tile 0 (one row a thread), 4-7 of row tile 1, 8 TMA, 9 MMA (10 and 11
// fill the warpgroup, whose registers the softmax warps take over: a row's 128 scores stay in
// registers).
// MMAs are issued in the order  PV_0(j-1) QK_0(j) PV_1(j-1) QK_1(j): they execute in order, so
// QK_i(j) may overwrite P_i(j-1), and when S_i(j) is complete so is O_i up to j-1.
//
// Softmax. The running maximum only has to keep the exponentials in range, so it is raised (and O
// rescaled) only when a tile exceeds it by more than 2^8; sums and O are fp32, and P carries the
// same relative rounding whatever its scale.
//
// What the cache holds beyond kv_len never enters a product: pages there are not read (TMA fills
// zeros for coordinates beyond the map), and the rest of the last page is zeroed in shared
// memory, since 0 * NaN in P V would not vanish.
#include "attn.h"
#include "tc_common.cuh"

namespace moe {
namespace {

using namespace ptx;
using tc::drain_bar;
using tc::wait_bar;

constexpr int kRows = 128;           // rows of a row tile (MMA M)
constexpr int kKeys = kPrefillKeys;  // places of a key tile
constexpr int kThreads = 384;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct PrefillParams {
  int T, B, Hq, Hkv, G, TQ;  // TQ: tokens of a row tile
  int page_size, max_pages, num_pages;
  int box_rows;              // rows of a cache box
  int max_len;               // places that the table can hold
  int window, n_sink;
  FastDiv page_div, g_div;
  float scale;
  int64_t o_stride;
  const int32_t* block_table;  // NULL: sequence b lies in page b
  const int32_t* kv_len;
  const int32_t* q_start;
  const float* k_scale;
  const float* v_scale;
  uint16_t* o;
  float* lse;
  int* status;
};

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;                    // 64-column boxes of a row
  static constexpr uint32_t kHalfBytes = kKeys * 128;       // 128 rows of 128 bytes
  static constexpr uint32_t kTileBytes = kHalves * kHalfBytes;
  static constexpr int kSlots = D == 128 ? 5 : 10;          // K and V tiles in flight
  static constexpr uint32_t kQBytes = 2 * kTileBytes;
  static constexpr uint32_t kSmem = kQBytes + kSlots * kTileBytes + 1024;
  static constexpr uint32_t kTmemO = 256;                   // columns: S0, S1, O0, O1
  static_assert(kSmem + 1024 <= 227 * 1024, "shared memory");
};

// The block's piece of work.
struct Work {
  int b, h;           // sequence, key head
  int tok0, ntok;     // first row of q, tokens (over both row tiles)
  int pos0;           // place of the first token
  int len;            // kv_len
  int sink_tiles;     // key tiles 0 .. that hold sinks
  int lo, n;          // first tile of the window; tiles to walk, sinks that lie before lo included
  int lead;           // of these, sink tiles before lo
};

// key tile of step j
__device__ __forceinline__ int key_tile(const Work& w, int j) {
  return j < w.lead ? j : w.lo + j - w.lead;
}

// first and last place of row tile i, and whether it sees anything of key tile kt
struct RowTile {
  int p0, p1;     // places of its first and last token
  int ntok;
  int lo, hi;     // key tiles of its window
};

__device__ __forceinline__ RowTile row_tile(const PrefillParams& p, const Work& w, int i) {
  RowTile r;
  r.ntok = min(p.TQ, w.ntok - i * p.TQ);
  r.p0 = w.pos0 + i * p.TQ;
  r.p1 = r.p0 + r.ntok - 1;
  r.lo = p.window ? max(0, r.p0 - p.window + 1) / kKeys : 0;
  r.hi = r.ntok > 0 && r.p1 >= 0 ? r.p1 / kKeys : -1;
  return r;
}

__device__ __forceinline__ bool sees(const RowTile& r, int sink_tiles, int kt) {
  return kt <= r.hi && (kt >= r.lo || kt < sink_tiles);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    k_attn_prefill(const __grid_constant__ CUtensorMap tm_q,
                   const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const PrefillParams p) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* q_s = smem;
  uint8_t* ring = smem + C::kQBytes;
  __shared__ uint64_t q_full[2], s_full[2], p_full[2], o_full[2], full[C::kSlots],
      empty[C::kSlots];
  __shared__ uint32_t tmem_holder;
  __shared__ int abort_flag_s;
  __shared__ Work work_s;
  volatile int* abort_flag = &abort_flag_s;
  const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);   // the row tile's four warps
      mbar_init(&o_full[i], 1);
    }
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    abort_flag_s = 0;
    fence_mbar_init();
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  if (warp == 9) {
    tmem_alloc(&tmem_holder, 512);
    tmem_relinquish();
  }
  pdl_wait_then_release();

  // ---- which sequence and which of its row tile pairs ----
  if (warp == 8) {
    const int pair_tok = 2 * p.TQ;
    int total = 0;  // pairs of all sequences
    const auto pairs_of = [&](int b, int& q0, int& n) {
      q0 = min(max(__ldg(p.q_start + b), 0), p.T);
      n = min(max(__ldg(p.q_start + b + 1), q0), p.T) - q0;
      return (n + pair_tok - 1) / pair_tok;
    };
    int q0, n;
    for (int b = lane; b < p.B; b += 32) total += pairs_of(b, q0, n);
#pragma unroll
    for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    // the last pairs of a sequence see the most keys: they start first
    const int want = total - 1 - (int)(blockIdx.x / (unsigned)p.Hkv);
    Work w{};
    w.b = -1;
    int before = 0;
    for (int b0 = 0; want >= 0 && b0 < p.B; b0 += 32) {
      const int b = b0 + lane;
      const int mine = b < p.B ? pairs_of(b, q0, n) : 0;
      int incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
      }
      const int all = __shfl_sync(0xffffffffu, incl, 31);
      if (want < before + all) {
        if (before + incl > want && before + incl - mine <= want) {
          const int pair = want - (before + incl - mine);
          w.b = b;
          w.h = (int)(blockIdx.x % (unsigned)p.Hkv);
          w.tok0 = q0 + pair * pair_tok;
          w.ntok = min(pair_tok, n - pair * pair_tok);
          int len = __ldg(p.kv_len + b);
          if (len < 0 || len > p.max_len) record_error(p.status, MOE_ERR_DEVICE_BOUNDS);
          len = min(max(len, 0), p.max_len);
          w.len = len;
          w.pos0 = len - n + pair * pair_tok;
          const int last = w.pos0 + w.ntok - 1;
          const int end = last >= 0 ? last / kKeys + 1 : 0;  // tiles up to the last token
          w.lo = p.window ? min(end, max(0, w.pos0 - p.window + 1) / kKeys) : 0;
          w.sink_tiles = (p.n_sink + kKeys - 1) / kKeys;
          w.lead = min(w.sink_tiles, w.lo);
          w.n = w.lead + end - w.lo;
          work_s = w;
        }
        break;
      }
      before += all;
    }
    const unsigned found = __ballot_sync(0xffffffffu, w.b >= 0);
    if (!found && lane == 0) {
      w.n = -1;
      work_s = w;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_holder;
  const Work w = work_s;

  // Registers: 384 threads of 168 at launch = 128 * (208 + 208 + 88).
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (w.n >= 0 && warp == 8) {
      // ---------------- TMA ----------------
      const uint64_t pol = policy_evict_normal();
      bool ok = true;
      int slot = 0, issued = 0;
      uint32_t phase = 0;
      if (lane == 0 && w.n > 0) {
        const uint32_t half_bytes = (uint32_t)(p.G * p.TQ) * 128;
        for (int i = 0; i < 2; ++i) {
          if (i * p.TQ >= w.ntok) break;
          mbar_arrive_expect_tx(&q_full[i], C::kHalves * half_bytes);
          for (int hf = 0; hf < C::kHalves; ++hf)
            tma_load_3d(q_s + i * C::kTileBytes + hf * C::kHalfBytes, &tm_q, &q_full[i], hf * 64,
                        w.h * p.G, w.tok0 + i * p.TQ, pol);
        }
      }
      // a lane's box of every tile: rows box * box_rows .., columns half * 64 ..
      const int boxes = kKeys / p.box_rows * C::kHalves;
      const int box = lane / C::kHalves, half = lane % C::kHalves;
      const int end = min(w.len, w.pos0 + w.ntok);                    // places any row sees
      const int lo = p.window ? max(0, w.pos0 - p.window + 1) : 0;
      for (int j = 0; ok && j < w.n; ++j) {
        const int key = key_tile(w, j) * kKeys + box * p.box_rows;
        int page = p.num_pages, row = 0;  // beyond the map: zeros
        if (lane < boxes && key < end && (key + p.box_rows > lo || key < p.n_sink)) {
          if (p.block_table) {
            const int pg = (int)div_fast((uint32_t)key, p.page_div);
            page = __ldg(p.block_table + (int64_t)w.b * p.max_pages + pg);
            row = key - pg * p.page_size;
            if ((uint32_t)page >= (uint32_t)p.num_pages) {
              record_error(p.status, MOE_ERR_DEVICE_BOUNDS);
              page = p.num_pages;
            }
          } else {
            page = w.b;
            row = key;
          }
        }
        for (int kv = 0; kv < 2; ++kv) {
          ok = wait_bar(&empty[slot], phase ^ 1u, abort_flag, p.status);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          ++issued;
          if (lane == 0) mbar_arrive_expect_tx(&full[slot], C::kTileBytes);
          __syncwarp();
          if (lane < boxes)
            tma_load_4d(ring + slot * C::kTileBytes + half * C::kHalfBytes +
                            box * p.box_rows * 128,
                        kv ? &tm_v : &tm_k, &full[slot], half * 64, row, w.h, page, pol);
          if (++slot == C::kSlots) { slot = 0; phase ^= 1u; }
        }
      }
      // every load issued has landed before the block may exit
      if (lane == 0) {
        for (int s = 0; s < C::kSlots; ++s) {
          if (s < issued) drain_bar(&full[s], s < slot ? phase : phase ^ 1u, p.status);
        }
        for (int i = 0; i < 2; ++i)
          if (w.n > 0 && i * p.TQ < w.ntok) drain_bar(&q_full[i], 0, p.status);
      }
    } else if (w.n > 0 && warp == 9) {
      // ---------------- MMA ----------------
      const RowTile rt[2] = {row_tile(p, w, 0), row_tile(p, w, 1)};
      const uint32_t idesc_s = idesc_bf16(kRows, kKeys), idesc_o = idesc_bf16_b_mn(kRows, D);
      const uint32_t q_u = smem_u32(q_s), ring_u = smem_u32(ring);
      uint32_t p_phase[2] = {0, 0};
      bool begun[2] = {false, false};
      const auto step_slot = [](int n, int& slot, uint32_t& phase) {
        slot = n % C::kSlots;
        phase = (uint32_t)(n / C::kSlots) & 1u;
      };
      bool ok = true;
      for (int i = 0; ok && i < 2; ++i)
        if (rt[i].ntok > 0) ok = wait_bar(&q_full[i], 0, abort_flag, p.status);
      ok = __all_sync(0xffffffffu, ok);
      for (int j = 0; ok && j <= w.n; ++j) {
        int ks = 0, vs = 0;
        uint32_t kp = 0, vp = 0;
        step_slot(2 * j, ks, kp);
        const int kt = j < w.n ? key_tile(w, j) : 0, vt = j > 0 ? key_tile(w, j - 1) : 0;
        if (j < w.n) ok = wait_bar(&full[ks], kp, abort_flag, p.status);
        if (ok && j > 0) {
          step_slot(2 * j - 1, vs, vp);
          ok = wait_bar(&full[vs], vp, abort_flag, p.status);
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (j > 0 && p.block_table && (vt + 1) * kKeys > w.len) {
          // the tile's places past kv_len: zeros, whatever their page holds
          const int r0 = w.len - vt * kKeys;
          for (int x = lane; x < (kKeys - r0) * 8 * C::kHalves; x += 32) {
            const int r = r0 + x / (8 * C::kHalves), c = x % (8 * C::kHalves);
            *reinterpret_cast<uint4*>(ring + vs * C::kTileBytes + (c >> 3) * C::kHalfBytes +
                                      r * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t s_t = tmem + i * kKeys, o_t = tmem + C::kTmemO + i * D;
          if (j > 0 && sees(rt[i], w.sink_tiles, vt)) {
            if (!wait_bar(&p_full[i], p_phase[i], abort_flag, p.status)) ok = false;
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            p_phase[i] ^= 1u;
            tc_fence_after();
            if (lane == 0) {
              const uint64_t dv = sw128_mn_desc(ring_u + vs * C::kTileBytes, C::kHalfBytes);
#pragma unroll
              for (int kk = 0; kk < kKeys / 16; ++kk)
                mma_ts(o_t, s_t + 8 * kk, dv + (uint64_t)(kk * (2048 >> 4)), idesc_o,
                       (begun[i] || kk) ? 1u : 0u);
              if (vt == rt[i].hi) mma_commit(&o_full[i]);  // its last
            }
            begun[i] = true;
          }
          if (j < w.n && sees(rt[i], w.sink_tiles, kt)) {
            if (lane == 0) {
              const uint64_t dq = sw128_desc(q_u + i * C::kTileBytes);
              const uint64_t dk = sw128_desc(ring_u + ks * C::kTileBytes);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint64_t at = (uint64_t)((kk >> 2) * (C::kHalfBytes >> 4) + (kk & 3) * 2);
                mma_bf16_ss(s_t, dq + at, dk + at, idesc_s, kk ? 1u : 0u);
              }
              mma_commit(&s_full[i]);
            }
          }
        }
        if (!ok) break;
        if (lane == 0) {
          if (j > 0) mma_commit(&empty[vs]);
          if (j < w.n) mma_commit(&empty[ks]);
        }
        __syncwarp();
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    if (w.n >= 0) {
      // ---------------- softmax and epilogue ----------------
      const int i = warp >> 2;
      const RowTile rt = row_tile(p, w, i);
      const int r = (warp & 3) * 32 + lane;                 // row of the tile
      const int t = (int)div_fast((uint32_t)r, p.g_div);    // its token
      const int pos = rt.p0 + t;
      const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
      const uint32_t s_t = lanes + i * kKeys, o_t = lanes + C::kTmemO + i * D;
      const float sc2 = p.scale * kLog2e * (p.k_scale ? __ldg(p.k_scale + w.h) : 1.f);
      float m = -INFINITY, l = 0.f;
      uint32_t phase = 0;
      bool ok = true, begun = false;
      for (int j = 0; ok && j < w.n; ++j) {
        const int kt = key_tile(w, j);
        if (!sees(rt, w.sink_tiles, kt)) continue;
        ok = wait_bar(&s_full[i], phase, abort_flag, p.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        phase ^= 1u;
        tc_fence_after();
        uint32_t s[kKeys];
#pragma unroll
        for (int c = 0; c < kKeys; c += 32) tmem_ld32(s_t + c, s + c);
#pragma unroll
        for (int c = 0; c < kKeys; c += 32) tmem_ld_wait32(s + c);
        const int k0 = kt * kKeys;
        const bool plain = k0 + kKeys - 1 <= rt.p0 &&
                           (!p.window || k0 > rt.p1 - p.window || k0 + kKeys <= p.n_sink);
        if (!plain) {
          const int hi = pos - k0;                                  // columns up to hi are seen
          const int lo = p.window ? hi - p.window : -1;             // and after lo
          const int sk = p.n_sink - k0;                             // or before sk
#pragma unroll
          for (int c = 0; c < kKeys; ++c)
            if (c > hi || (c <= lo && c >= sk)) s[c] = 0xFF800000u;
        }
        float mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < kKeys; ++c) mx = fmaxf(mx, __uint_as_float(s[c]));
        // raise the running maximum only where it is exceeded by 2^8 (or has no value yet)
        const bool raise = mx > m && (m == -INFINITY || (mx - m) * sc2 > 8.f);
        const float f = raise && m != -INFINITY ? ex2((m - mx) * sc2) : 1.f;
        if (raise) {
          l = m == -INFINITY ? 0.f : l * f;
          m = mx;
        }
        if (begun && __any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll
          for (int c = 0; c < D; c += 32) {
            uint32_t y[32];
            tmem_ld32(o_t + c, y);
            tmem_ld_wait32(y);
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * f);
            tmem_st32(o_t + c, y);
          }
        }
        begun = true;
        const float base = m == -INFINITY ? 0.f : m * sc2;
        float sum = 0.f;
#pragma unroll
        for (int c = 0; c < kKeys; c += 64) {
          uint32_t pk[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float e0 = ex2(fmaf(__uint_as_float(s[c + 2 * e]), sc2, -base));
            const float e1 = ex2(fmaf(__uint_as_float(s[c + 2 * e + 1]), sc2, -base));
            sum += e0 + e1;
            pk[e] = pack_bf16(e0, e1);
          }
          tmem_st32(s_t + (c >> 1), pk);
        }
        l += sum;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[i]);
      }
      if (begun && ok) ok = __all_sync(0xffffffffu, wait_bar(&o_full[i], 0, abort_flag, p.status));
      if (ok) {
        tc_fence_after();
        const bool mine = r < p.G * p.TQ && t < rt.ntok;
        const int64_t tok = w.tok0 + i * p.TQ + t;
        const int head = w.h * p.G + (r - t * p.G);
        const float vsc = p.v_scale ? __ldg(p.v_scale + w.h) : 1.f;
        const float inv = l == 0.f ? 0.f : vsc / l;
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          uint32_t y[32];
          if (begun) {
            tmem_ld32(o_t + c, y);
            tmem_ld_wait32(y);
          }
          if (mine) {
            uint4* dst = reinterpret_cast<uint4*>(p.o + tok * p.o_stride + (int64_t)head * D + c);
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              uint32_t z[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                z[k] = inv == 0.f ? 0u
                                  : pack_bf16(__uint_as_float(y[e + 2 * k]) * inv,
                                              __uint_as_float(y[e + 2 * k + 1]) * inv);
              dst[e / 8] = make_uint4(z[0], z[1], z[2], z[3]);
            }
          }
        }
        if (mine && p.lse)
          p.lse[tok * p.Hq + head] = l == 0.f ? -INFINITY : m * sc2 * kLn2 + logf(l);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---- caches that the tiles cannot read as they lie ---------------------------------------------
// Copies what this step's tokens see into rows in order: E4M3 codes become bf16 exactly (the
// scales stay outside), and places that no token sees but that share a tile with one are zeros.
// Bound by HBM: one read of the visible cache and one bf16 write, against 2 G n D flops an
// element for n tokens a sequence.
template <int D, bool FP8>
__global__ void __launch_bounds__(256) k_attn_unpack(const AttnDims a, const uint8_t* k_cache,
                                                     const uint8_t* v_cache,
                                                     const int32_t* block_table,
                                                     const int32_t* kv_len,
                                                     const int32_t* q_start, uint16_t* out,
                                                     int64_t lp, int* status) {
  constexpr int CH = D / 8;  // 8 elements a thread
  const int h = (int)blockIdx.y, k0 = (int)blockIdx.x * kKeys;
  pdl_wait_then_release();
  for (int b = (int)blockIdx.z; b < a.B; b += (int)gridDim.z) {
    const int len = min(max(__ldg(kv_len + b), 0), a.max_pages * a.page_size);
    const int n = __ldg(q_start + b + 1) - __ldg(q_start + b);
    if (n <= 0 || k0 >= len) continue;
    const int lo = a.window ? max(0, len - n - a.window + 1) : 0;
    if (k0 + kKeys <= lo && k0 >= a.n_sink) continue;
    const int64_t half = (int64_t)a.B * a.Hkv * lp * D;
    for (int x = (int)threadIdx.x; x < kKeys * CH; x += 256) {
      const int j = k0 + x / CH, c = x % CH;
      uint4 kv[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
      if (j < len && (j >= lo || j < a.n_sink)) {
        const int pg = (int)div_fast((uint32_t)j, a.page_div);
        const int page = __ldg(block_table + (int64_t)b * a.max_pages + pg);
        if ((uint32_t)page >= (uint32_t)a.num_pages) {
          record_error(status, MOE_ERR_DEVICE_BOUNDS);
        } else {
          const int64_t at = (int64_t)page * a.page_stride + (int64_t)h * a.head_stride +
                             (int64_t)(j - pg * a.page_size) * a.token_stride + c * 8;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint8_t* src = i ? v_cache : k_cache;
            if (FP8) {
              const uint2 u = *reinterpret_cast<const uint2*>(src + at);
              uint32_t z[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t w = e < 2 ? u.x : u.y;
                uint32_t f;
                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f) : "h"((uint16_t)(w >> (16 * (e & 1)))));
                float x0, x1;
                asm("{.reg .b16 lo, hi; mov.b32 {lo, hi}, %2; cvt.f32.f16 %0, lo; "
                    "cvt.f32.f16 %1, hi;}" : "=f"(x0), "=f"(x1) : "r"(f));
                z[e] = pack_bf16(x0, x1);
              }
              kv[i] = make_uint4(z[0], z[1], z[2], z[3]);
            } else {
              kv[i] = *reinterpret_cast<const uint4*>(src + 2 * at);
            }
          }
        }
      }
      uint16_t* dst = out + (((int64_t)b * a.Hkv + h) * lp + j) * D + c * 8;
      *reinterpret_cast<uint4*>(dst) = kv[0];
      *reinterpret_cast<uint4*>(dst + half) = kv[1];
    }
  }
}

cudaError_t encode_bf16(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims,
                        const cuuint64_t* strides, const cuuint32_t* box) {
  tc::EncodeTiledFn fn = tc::encode_fn();
  if (!fn) return cudaErrorNotSupported;
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank,
                        const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D>
cudaError_t launch(const AttnDims& a, const void* q, const void* k, const void* v,
                   PrefillParams& p, int64_t page_stride, int64_t head_stride,
                   int64_t token_stride, cudaStream_t st) {
  using C = Cfg<D>;
  p.TQ = kRows / a.G;
  CUtensorMap mq, mk, mv;
  {
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a.Hq, (cuuint64_t)a.T};
    const cuuint64_t str[2] = {(cuuint64_t)D * 2, (cuuint64_t)a.qr_stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)a.G, (cuuint32_t)p.TQ};
    cudaError_t e = encode_bf16(&mq, q, 3, dims, str, box);
    if (e != cudaSuccess) return e;
  }
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)p.page_size, (cuuint64_t)a.Hkv,
                              (cuuint64_t)p.num_pages};
  const cuuint64_t str[3] = {(cuuint64_t)token_stride * 2, (cuuint64_t)head_stride * 2,
                             (cuuint64_t)page_stride * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)p.box_rows, 1, 1};
  cudaError_t e = encode_bf16(&mk, k, 4, dims, str, box);
  if (e == cudaSuccess) e = encode_bf16(&mv, v, 4, dims, str, box);
  if (e != cudaSuccess) return e;
  auto kern = k_attn_prefill<D>;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
  if (e != cudaSuccess) return e;
  // row tile pairs: sum over sequences of ceil(n / pair) <= T / pair + B, and <= T
  const int64_t most = (int64_t)a.T / (2 * p.TQ) + a.B;
  const unsigned pairs = (unsigned)(most < a.T ? most : a.T);  // times Hkv: under 2^31 (host check)
  count_launches(1);
  return launch_pdl(kern, dim3(pairs * (unsigned)a.Hkv), dim3(kThreads), C::kSmem, st, mq, mk, mv,
                    p);
}

template <int D>
cudaError_t launch_unpack(const AttnDims& a, const void* k, const void* v, const int32_t* table,
                          const int32_t* kv_len, const int32_t* q_start, void* out, int64_t lp,
                          int* status, cudaStream_t st) {
  const dim3 grid((unsigned)(lp / kKeys), (unsigned)a.Hkv, (unsigned)(a.B < 65535 ? a.B : 65535));
  auto kern = a.fp8 ? k_attn_unpack<D, true> : k_attn_unpack<D, false>;
  count_launches(1);
  return launch_pdl(kern, grid, dim3(256), 0, st, a, static_cast<const uint8_t*>(k),
                    static_cast<const uint8_t*>(v), table, kv_len, q_start,
                    static_cast<uint16_t*>(out), lp, status);
}

}  // namespace

cudaError_t launch_attn_prefill(const AttnDims& a, const void* q, const void* k_cache,
                                const void* v_cache, const float* k_scale, const float* v_scale,
                                const int32_t* block_table, const int32_t* kv_len,
                                const int32_t* q_start, void* o, float* lse, char* ws,
                                const AttnWs& L, cudaStream_t st) {
  PrefillParams p{};
  p.T = a.T;
  p.B = a.B;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.G = a.G;
  p.max_len = a.max_pages * a.page_size;
  p.window = a.window;
  p.n_sink = a.n_sink;
  p.g_div = fast_div((uint32_t)a.G);
  p.scale = a.scale;
  p.o_stride = a.o_stride;
  p.kv_len = kv_len;
  p.q_start = q_start;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.o = static_cast<uint16_t*>(o);
  p.lse = lse;
  p.status = reinterpret_cast<int*>(ws + L.status);
  p.max_pages = a.max_pages;
  int64_t ps = a.page_stride, hs = a.head_stride, ts = a.token_stride;
  if (prefill_reads_pages(a)) {
    p.block_table = block_table;
    p.page_size = a.page_size;
    p.num_pages = a.num_pages;
    p.page_div = a.page_div;
    p.box_rows = a.page_size < kKeys ? a.page_size : kKeys;
  } else {
    const int64_t lp = unpacked_len(a);
    void* out = ws + L.unpacked;
    cudaError_t e = a.D == 64 ? launch_unpack<64>(a, k_cache, v_cache, block_table, kv_len,
                                                  q_start, out, lp, p.status, st)
                              : launch_unpack<128>(a, k_cache, v_cache, block_table, kv_len,
                                                   q_start, out, lp, p.status, st);
    if (e != cudaSuccess) return e;
    ts = a.D;
    hs = lp * a.D;
    ps = hs * a.Hkv;
    k_cache = out;
    v_cache = ws + L.unpacked + (size_t)a.B * ps * 2;
    p.block_table = nullptr;
    p.page_size = (int)lp;
    p.num_pages = a.B;
    p.page_div = fast_div(1);
    p.box_rows = kKeys;
  }
  return a.D == 64 ? launch<64>(a, q, k_cache, v_cache, p, ps, hs, ts, st)
                   : launch<128>(a, q, k_cache, v_cache, p, ps, hs, ts, st);
}

}  // namespace moe
