// Attention of any number of new tokens per sequence over the paged cache (prompts, and chunks of
// prompts), on tcgen05 tensor cores.
//
//   s_ij = scale q_i.k_j over the places j that token i sees, o_i = sum_j softmax(s_i)_j v_j
//
// What bounds it: the tensor cores, 4 D flops per visible (query head, key) pair; next to them
// the exponentials, one per pair, and the shared-memory and L2 bandwidth that the operands take.
//
// Tiles. The G query heads of a key head share its keys, so a tile of 128 rows is 128/G
// consecutive tokens times G heads (row t*G + g; when G does not divide 128 the last rows are
// idle), and the key axis runs in tiles of 64 places. A block holds two row tiles of one sequence
// and key head and walks the key tiles that any of their rows sees: the sinks, then from the
// window's first place to the last token. While the softmax works on one row tile's scores the
// tensor cores work on the other's.
//
// Heads of 128 run on pairs of blocks (cta_group::2): row tile i of the pair is 256 rows, 128 in
// each block; each block loads half of a key tile (32 places of K, 64 columns of V) and one MMA of
// M = 256 reads both halves, which halves the traffic of K and V from L2 and through shared
// memory. Heads of 64 are bound by the exponentials before that and run on single blocks.
//
// Tensor memory: per row tile two buffers of 64 columns of scores S (fp32) and D columns of output
// O (fp32). The probabilities P (bf16) overwrite their S and are the A operand of the second
// product from there; K is K-major and V MN-major as TMA lays both down (rows of places, 128-byte
// swizzle).
//
// Warps: 0-3 softmax of row tile 0 (one row a thread), 4-7 of row tile 1, 8 TMA of Q and K, 10 of
// V, 9 and 11 the MMAs of row tiles 0 and 1 (in the pair's even block). One warp for all four
// would be too slow: a tile takes the tensor cores about 1000 cycles, and each warp's share of
// waits, look-ups and issues 200 to 500. The last warpgroup's registers go to the softmax warps.
// A row tile's MMAs are issued in the order  QK(0) QK(1) PV(0) QK(2) PV(1) ...  and execute in
// order: S(j+1) is formed while the softmax works on S(j), and QK(j+1) may overwrite P(j-1).
//
// Softmax. The row maximum of a tile that needs no mask comes with its load (tcgen05.ld.red). The
// running maximum only has to keep the exponentials in range, so it is raised (and O rescaled)
// only when a tile exceeds it by more than 2^8; sums and O are fp32, and P carries the same
// relative rounding whatever its scale.
//
// What the cache holds beyond kv_len never enters a product: pages there are not read (TMA fills
// zeros for coordinates beyond the map), and the rest of the last page is zeroed in shared
// memory, since 0 * NaN in P V would not vanish.
#include <type_traits>

#include "attn.h"
#include "tc_common.cuh"

namespace moe {
namespace {

using namespace ptx;
using tc::drain_bar;

constexpr int kRows = 128;           // rows of a block's row tile
constexpr int kKeys = 64;            // places of a key tile
constexpr int kThreads = 384;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kNoMax = -3e38f;     // the maximum of no scores: finite, so that -inf - it is -inf

struct PrefillParams {
  int T, B, Hq, Hkv, G, TQ;  // TQ: tokens of a block's row tile
  int page_size, max_pages, num_pages;
  int k_rows, v_rows;        // places of a box of K, of V
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
  static constexpr bool kPair = D == 128;
  static constexpr int kBlocks = kPair ? 2 : 1;             // blocks that share a key tile
  static constexpr int kHalves = D / 64;                    // 64-column boxes of a row of Q
  static constexpr uint32_t kHalfBytes = kRows * 128;       // 128 rows of 128 bytes
  static constexpr uint32_t kQTile = kHalves * kHalfBytes;
  // a block's part of a K or V tile: 32 places x 128 columns of K, 64 places x 64 columns of V
  // (pairs), or 64 places x 64 columns
  static constexpr uint32_t kSlot = kKeys * 128;
  static constexpr uint32_t kKHalf = kSlot / kHalves;       // K: bytes of a 64-column half
  static constexpr int kSlots = 10;                         // of K, and of V
  static constexpr uint32_t kQBytes = 2 * kQTile;
  static constexpr uint32_t kSmem = kQBytes + 2 * kSlots * kSlot + 1024;
  static constexpr uint32_t kTmemO = 256;  // columns: S of row tile 0 (two buffers), of 1; O0, O1
  static_assert(kSmem + 1024 <= 227 * 1024, "shared memory");
};

// two fp32 in a 64-bit register: one instruction for both
__device__ __forceinline__ uint64_t f32x2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void f32x2_split(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// The piece of work of a block, or of a pair.
struct Work {
  int b, h;           // sequence, key head
  int tok0, ntok;     // first row of q, tokens (over all row tiles)
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

// Tokens [first, first + span) of the work: the places p0 .. p1 of the first and the last of them,
// and the steps [0, sink) and [from, to) whose key tiles any of them sees.
struct RowTile {
  int p0, p1, ntok;
  int sink, from, to;
};

__device__ __forceinline__ RowTile row_tile(const PrefillParams& p, const Work& w, int first,
                                            int span) {
  RowTile r;
  r.ntok = min(span, w.ntok - first);
  r.p0 = w.pos0 + first;
  r.p1 = r.p0 + r.ntok - 1;
  const bool any = r.ntok > 0 && r.p1 >= 0;
  const int lo = p.window ? max(0, r.p0 - p.window + 1) / kKeys : 0;
  const int skip = w.lo - w.lead;  // tiles between the sinks' and the window's
  r.to = any ? r.p1 / kKeys + 1 - skip : 0;
  // sink tiles past the window's first are among its steps
  r.sink = min(r.to, w.sink_tiles > w.lo ? w.sink_tiles - skip : w.lead);
  r.from = min(r.to, max(r.sink, lo - skip));
  return r;
}

__device__ __forceinline__ bool sees(const RowTile& r, int j) {
  return j < r.sink || (j >= r.from && j < r.to);
}

// Bounded wait on an mbarrier phase: false (after recording a timeout) if it gave up or another
// role did. The clock is read only after 64 tries: reading it costs more than most waits last.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                         int* status) {
  for (int i = 0; i < 64; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return tc::wait_bar(bar, parity, abort_flag, status);
}

// wait_bar for a barrier that the other block of the pair arrives on as well
__device__ __forceinline__ bool wait_bar_pair(uint64_t* bar, uint32_t parity,
                                              volatile int* abort_flag, int* status) {
  return wait_bar(bar, parity, abort_flag, status) && mbar_try_wait_cluster(bar, parity);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    k_attn_prefill(const __grid_constant__ CUtensorMap tm_q,
                   const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const PrefillParams p) {
  using C = Cfg<D>;
  constexpr bool PAIR = C::kPair;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* q_s = smem;
  uint8_t* ring = smem + C::kQBytes;
  // q_full, full, p_full and tail_ready are waited on in the pair's even block
  __shared__ uint64_t q_full[2], s_full[2][2], p_full[2][2], o_full[2], o_done[2], tail_full,
      tail_ready, full[2][C::kSlots], empty[2][C::kSlots];  // of K, of V
  __shared__ uint32_t tmem_holder;
  __shared__ int abort_flag_s;
  __shared__ Work work_s;
  volatile int* abort_flag = &abort_flag_s;
  const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31;
  const int rank = PAIR ? (int)cluster_ctarank() : 0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&o_full[i], 1);                       // a phase for every PV
      mbar_init(&o_done[i], 1);                       // the last one
      for (int b = 0; b < 2; ++b) {
        mbar_init(&s_full[i][b], 1);
        mbar_init(&p_full[i][b], 4 * C::kBlocks);     // the row tile's warps
      }
    }
    mbar_init(&tail_full, 1);
    mbar_init(&tail_ready, C::kBlocks);
    for (int s = 0; s < C::kSlots; ++s) {
      for (int kv = 0; kv < 2; ++kv) {
        mbar_init(&full[kv][s], 1);
        mbar_init(&empty[kv][s], 2);  // both row tiles' MMAs have read it
      }
    }
    abort_flag_s = 0;
    fence_mbar_init();
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  if (warp == 9) {
    if (PAIR) {
      tmem_alloc_pair(&tmem_holder, 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(&tmem_holder, 512);
      tmem_relinquish();
    }
  }
  pdl_wait_then_release();

  // ---- which sequence and which of its row tiles ----
  const int span = p.TQ * C::kBlocks;  // tokens of a row tile of the work
  if (warp == 8) {
    const int unit_tok = 2 * span;
    const int unit = (int)blockIdx.x / C::kBlocks;
    int total = 0;  // units of all sequences
    const auto units_of = [&](int b, int& q0, int& n) {
      q0 = min(max(__ldg(p.q_start + b), 0), p.T);
      n = min(max(__ldg(p.q_start + b + 1), q0), p.T) - q0;
      return (n + unit_tok - 1) / unit_tok;
    };
    int q0, n;
    for (int b = lane; b < p.B; b += 32) total += units_of(b, q0, n);
#pragma unroll
    for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    // the last units of a sequence see the most keys: they start first
    const int want = total - 1 - unit / p.Hkv;
    Work w{};
    w.b = -1;
    int before = 0;
    for (int b0 = 0; want >= 0 && b0 < p.B; b0 += 32) {
      const int b = b0 + lane;
      const int mine = b < p.B ? units_of(b, q0, n) : 0;
      int incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
      }
      const int all = __shfl_sync(0xffffffffu, incl, 31);
      if (want < before + all) {
        if (before + incl > want && before + incl - mine <= want) {
          const int at = (want - (before + incl - mine)) * unit_tok;
          w.b = b;
          w.h = unit % p.Hkv;
          w.tok0 = q0 + at;
          w.ntok = min(unit_tok, n - at);
          int len = __ldg(p.kv_len + b);
          if (len < 0 || len > p.max_len) record_error(p.status, MOE_ERR_DEVICE_BOUNDS);
          len = min(max(len, 0), p.max_len);
          w.len = len;
          w.pos0 = len - n + at;
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
  if (PAIR) cluster_sync();  // both blocks' barriers are initialised
  tc_fence_after();
  const uint32_t tmem = tmem_holder;
  const Work w = work_s;
  // places past kv_len share the last tile (of a cache read in place) with some before it
  const bool tail = w.n > 0 && p.block_table && (key_tile(w, w.n - 1) + 1) * kKeys > w.len;

  // Registers: 384 threads of 168 at launch = 128 * (200 + 200 + 104).
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (w.n > 0 && (warp == 8 || warp == 10)) {
      // ---------------- TMA: warp 8 Q and K, warp 10 V (one thread each) ----------------
      const int kv = warp == 8 ? 0 : 1;
      const uint32_t ring_kv = smem_u32(ring) + kv * (C::kSlots * C::kSlot);
      if (elect_one()) {
        if (kv == 0) {
          const uint32_t bytes = C::kHalves * (uint32_t)(p.G * p.TQ) * 128;
          for (int i = 0; i < 2; ++i) {
            if (i * span >= w.ntok) break;
            if (rank == 0) mbar_arrive_expect_tx(&q_full[i], C::kBlocks * bytes);
            const uint32_t bar =
                PAIR ? mapa_shared(smem_u32(&q_full[i]), 0) : smem_u32(&q_full[i]);
            for (int hf = 0; hf < C::kHalves; ++hf)
              tma_load_3d<PAIR>(smem_u32(q_s) + i * C::kQTile + hf * C::kHalfBytes, &tm_q, bar,
                                hf * 64, w.h * p.G, w.tok0 + i * span + rank * p.TQ);
          }
        }
        // A tile's boxes: rows box * rows .. of this block's part. K of a pair: its 32 places, both
        // 64-column halves (in one box if that takes all 32, else box by box); V of a pair: all 64
        // places of its half; else all 64 places.
        constexpr int kKRows = kKeys / C::kHalves;
        const int rows = kv ? p.v_rows : p.k_rows;
        const int part = kv ? kKeys : kKRows;                 // places of the block's part
        const bool split = kv == 0 && PAIR && rows < kKRows;  // halves in boxes of their own
        const int first = kv ? 0 : rank * kKRows;             // its first place of a tile
        const int half = kv && PAIR ? rank : 0;
        const int end = min(w.len, w.pos0 + w.ntok);          // places any row sees
        const int lo = p.window ? max(0, w.pos0 - p.window + 1) : 0;
        const int32_t* table = p.block_table + (int64_t)w.b * p.max_pages;
        const CUtensorMap* map = kv ? &tm_v : &tm_k;
        const uint32_t full_bar = PAIR ? mapa_shared(smem_u32(&full[kv][0]), 0)
                                       : smem_u32(&full[kv][0]);
        // page and row of the box at place `key`; the page is beyond the map, which reads as zeros,
        // if no row sees the box
        const auto look_up = [&](int key, int& page, int& row) {
          page = p.num_pages;
          row = 0;
          if (key >= end || (key + rows <= lo && key >= p.n_sink)) return;
          const int pg = p.block_table ? (int)div_fast((uint32_t)key, p.page_div) : w.b;
          row = p.block_table ? key - pg * p.page_size : key;
          page = pg;
          if (p.block_table) {
            page = __ldg(table + pg);
            if ((uint32_t)page >= (uint32_t)p.num_pages) {
              record_error(p.status, MOE_ERR_DEVICE_BOUNDS);
              page = p.num_pages;
            }
          }
        };
        // the boxes of tile j into a slot, completing on `bar`; the first one's page is known
        const auto load = [&](int j, uint32_t dst, uint32_t bar, int page, int row, auto pair) {
          constexpr bool P = decltype(pair)::value;
          tma_load_5d<P>(dst, map, bar, 0, row, half, w.h, page);
          if (split) tma_load_5d<P>(dst + C::kKHalf, map, bar, 0, row, 1, w.h, page);
          for (int r = rows; r < part; r += rows) {
            look_up(key_tile(w, j) * kKeys + first + r, page, row);
            tma_load_5d<P>(dst + r * 128, map, bar, 0, row, half, w.h, page);
            if (split) tma_load_5d<P>(dst + C::kKHalf + r * 128, map, bar, 0, row, 1, w.h, page);
          }
        };
        int page, row;  // of the next tile's first box: looked up a step before they are used
        look_up(key_tile(w, 0) * kKeys + first, page, row);
        // the last V tile is completed in shared memory if it ends past kv_len
        const int n = w.n - (kv == 1 && tail ? 1 : 0);
        bool ok = true;
        int slot = 0, issued = 0;
        uint32_t phase = 0;
        for (; issued < n; ++issued) {
          ok = wait_bar(&empty[kv][slot], phase ^ 1u, abort_flag, p.status);
          if (!ok) break;
          if (rank == 0) mbar_arrive_expect_tx(&full[kv][slot], C::kBlocks * C::kSlot);
          const int pg = page, rw = row;
          load(issued, ring_kv + slot * C::kSlot, full_bar + 8 * slot, pg, rw,
               std::integral_constant<bool, PAIR>());
          if (issued + 1 < w.n) look_up(key_tile(w, issued + 1) * kKeys + first, page, row);
          if (++slot == C::kSlots) { slot = 0; phase ^= 1u; }
        }
        if (ok && n < w.n) {
          ok = wait_bar(&empty[kv][slot], phase ^ 1u, abort_flag, p.status);
          if (ok) {
            mbar_arrive_expect_tx(&tail_full, C::kSlot);
            if (rank == 0) mbar_arrive(&full[kv][slot]);
            load(n, ring_kv + slot * C::kSlot, smem_u32(&tail_full), page, row,
                 std::integral_constant<bool, false>());
            ++issued;
            if (++slot == C::kSlots) { slot = 0; phase ^= 1u; }
          }
        }
        // every load issued has landed before the block may exit (in pairs the even block's
        // barriers count both blocks' bytes)
        if (rank == 0) {
          for (int s = 0; s < C::kSlots; ++s)
            if (s < issued) drain_bar(&full[kv][s], s < slot ? phase : phase ^ 1u, p.status);
          if (kv == 0)
            for (int i = 0; i < 2; ++i)
              if (i * span < w.ntok) drain_bar(&q_full[i], 0, p.status);
        }
        if (kv == 1 && tail && issued == w.n) drain_bar(&tail_full, 0, p.status);
      }
      __syncwarp();
      if (kv == 0 && tail) {
        // the places of the last V tile past kv_len: zeros
        bool ok = wait_bar(&tail_full, 0, abort_flag, p.status);
        ok = __all_sync(0xffffffffu, ok);
        if (ok) {
          const int r0 = w.len - key_tile(w, w.n - 1) * kKeys;
          uint8_t* vt = ring + (C::kSlots + (w.n - 1) % C::kSlots) * C::kSlot;
          for (int x = lane; x < (kKeys - r0) * 8; x += 32)
            *reinterpret_cast<uint4*>(vt + (r0 + x / 8) * 128 + (x & 7) * 16) =
                make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (PAIR)
              mbar_arrive_release_cluster(mapa_shared(smem_u32(&tail_ready), 0));
            else
              mbar_arrive(&tail_ready);
          }
        }
      }
    } else if (w.n > 0 && (warp == 9 || warp == 11) && rank == 0) {
      // ---------------- MMA: warp 9 row tile 0, warp 11 row tile 1 (one thread each) ----------------
      const int i = warp == 9 ? 0 : 1;
      const RowTile rt = row_tile(p, w, i * span, span);
      const uint32_t idesc_s = idesc_bf16(kRows * C::kBlocks, kKeys);
      const uint32_t idesc_o = idesc_bf16_b_mn(kRows * C::kBlocks, D);
      const uint32_t s_t = tmem + i * 2 * kKeys, o_t = tmem + C::kTmemO + i * D;
      const uint64_t dq = sw128_desc(smem_u32(q_s) + i * C::kQTile);
      const uint64_t dk0 = sw128_desc(smem_u32(ring));
      const uint64_t dv0 = sw128_mn_desc(smem_u32(ring) + C::kSlots * C::kSlot, C::kSlot);
      const auto commit = [&](uint64_t* bar) {
        if (PAIR)
          mma_commit_pair(bar);
        else
          mma_commit(bar);
      };
      if (elect_one()) {
        int n_qk = 0, n_pv = 0;  // products issued: the buffer and phase of the next
        int ks = 0, vs = 0;      // slots of the next K and V tile
        uint32_t kp = 0, vp = 0;
        // S = Q K(j); the K tile has arrived
        const auto qk = [&](int j) {
          if (!sees(rt, j)) return;
          const uint64_t dk = dk0 + (uint64_t)(ks * (int)(C::kSlot >> 4));
          const uint32_t d = s_t + (n_qk & 1) * kKeys;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t qa = dq + (uint64_t)((kk >> 2) * (C::kHalfBytes >> 4) + (kk & 3) * 2);
            const uint64_t ka = dk + (uint64_t)((kk >> 2) * (C::kKHalf >> 4) + (kk & 3) * 2);
            if (PAIR)
              mma_ss_pair(d, qa, ka, idesc_s, kk ? 1u : 0u);
            else
              mma_bf16_ss(d, qa, ka, idesc_s, kk ? 1u : 0u);
          }
          commit(&s_full[i][n_qk & 1]);
          ++n_qk;
        };
        // hands a slot back, also where the row tile saw nothing of its tile
        const auto free_k = [&] {
          commit(&empty[0][ks]);
          if (++ks == C::kSlots) { ks = 0; kp ^= 1u; }
        };
        bool ok = rt.ntok <= 0 || wait_bar(&q_full[i], 0, abort_flag, p.status);
        for (int j = 0; ok && j < min(2, w.n); ++j) {
          ok = wait_bar(&full[0][ks], kp, abort_flag, p.status);
          if (!ok) break;
          tc_fence_after();
          qk(j);
          free_k();
        }
        for (int j = 0; ok && j < w.n; ++j) {
          const bool more = j + 2 < w.n, pv = sees(rt, j);
          // the operands first: once P is there, nothing else holds up the products
          ok = wait_bar(&full[1][vs], vp, abort_flag, p.status);
          if (ok && tail && j + 1 == w.n) ok = wait_bar_pair(&tail_ready, 0, abort_flag, p.status);
          if (ok && more) ok = wait_bar(&full[0][ks], kp, abort_flag, p.status);
          if (ok && pv) ok = wait_bar(&p_full[i][n_pv & 1], (n_pv >> 1) & 1, abort_flag, p.status);
          if (!ok) break;
          tc_fence_after();
          if (pv) {  // O += P V(j)
            const uint64_t dv = dv0 + (uint64_t)(vs * (int)(C::kSlot >> 4));
            const uint32_t pa = s_t + (n_pv & 1) * kKeys;
#pragma unroll
            for (int kk = 0; kk < kKeys / 16; ++kk) {
              const uint64_t at = dv + (uint64_t)(kk * (2048 >> 4));
              const uint32_t acc = (n_pv || kk) ? 1u : 0u;
              if (PAIR)
                mma_ts_pair(o_t, pa + 8 * kk, at, idesc_o, acc);
              else
                mma_ts(o_t, pa + 8 * kk, at, idesc_o, acc);
            }
            ++n_pv;
          }
          if (more) qk(j + 2);
          if (pv) commit(&o_full[i]);
          if (j + 1 == rt.to) commit(&o_done[i]);
          commit(&empty[1][vs]);
          if (++vs == C::kSlots) { vs = 0; vp ^= 1u; }
          if (more) free_k();
        }
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    if (w.n >= 0) {
      // ---------------- softmax and epilogue ----------------
      const int i = warp >> 2;
      const RowTile both = row_tile(p, w, i * span, span);  // the row tile over all blocks
      const RowTile rt = row_tile(p, w, i * span + rank * p.TQ, p.TQ);
      const int r = (warp & 3) * 32 + lane;                 // row of the tile
      const int t = (int)div_fast((uint32_t)r, p.g_div);    // its token
      const int pos = rt.p0 + t;
      const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
      const uint32_t o_t = lanes + C::kTmemO + i * D;
      const uint32_t p_bar = PAIR ? mapa_shared(smem_u32(&p_full[i][0]), 0) : 0;
      const float sc2 = p.scale * kLog2e * (p.k_scale ? __ldg(p.k_scale + w.h) : 1.f);
      // the running maximum and sum, the maximum as a base-2 exponent
      float m = kNoMax, l = 0.f;
      int n = 0;  // tiles done
      bool ok = true;
      // key tiles whose every place every row sees: the first ones to, and of these those from (or
      // of sinks alone)
      const int plain_to = (rt.p0 + 1) / kKeys;
      const int plain_from = p.window ? max(0, rt.p1 - p.window + kKeys) / kKeys : 0;
      const int plain_sink = p.n_sink / kKeys;
      for (int j = both.sink ? 0 : both.from; ok && j < both.to;
           j = j + 1 == both.sink ? both.from : j + 1) {
        const int kt = key_tile(w, j);
        const int k0 = kt * kKeys;
        const bool plain = kt < plain_to && (kt >= plain_from || kt < plain_sink);
        ok = wait_bar(&s_full[i][n & 1], (n >> 1) & 1, abort_flag, p.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t s_t = lanes + (2 * i + (n & 1)) * kKeys;
        uint32_t s[kKeys];
        float mx2[2];
        tmem_ld_max32(s_t, s, mx2[0]);
        tmem_ld_max32(s_t + 32, s + 32, mx2[1]);
        tmem_ld_max_wait32(s, mx2[0]);
        tmem_ld_max_wait32(s + 32, mx2[1]);
        if (!plain) {
          asm volatile("" ::: "memory");  // a branch: predicated, the selects would cost every tile
          const int hi = pos - k0;                                  // columns up to hi are seen
          const int lo = p.window ? hi - p.window : -1;             // and after lo
          const int sk = p.n_sink - k0;                             // or before sk
#pragma unroll
          for (int c = 0; c < kKeys; ++c)
            if (c > hi || (c <= lo && c >= sk)) s[c] = 0xFF800000u;
          mx2[0] = mx2[1] = -INFINITY;
#pragma unroll
          for (int c = 0; c < kKeys; ++c) mx2[c & 1] = fmaxf(mx2[c & 1], __uint_as_float(s[c]));
        }
        const float mx = fmaxf(mx2[0], mx2[1]) * sc2;
        // raise the running maximum only where it is exceeded by 2^8 (or has no value yet)
        const bool raise = mx > m + 8.f;
        if (__any_sync(0xffffffffu, raise)) {
          const float f = raise ? ex2(m - mx) : 1.f;
          if (raise) m = mx;
          l *= f;
          if (n) {
            ok = wait_bar(&o_full[i], (n - 1) & 1, abort_flag, p.status);  // PV of the tile before
            // (S of this tile came after the PV before that one: the phase is unambiguous)
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              uint32_t y[16];
              tmem_ld16(o_t + c, y);
              tmem_ld_wait(y);
#pragma unroll
              for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * f);
              tmem_st16(o_t + c, y);
            }
          }
        }
        const uint64_t sc2x2 = f32x2(sc2, sc2), base2 = f32x2(-m, -m);
        uint64_t sum2[2] = {0, 0};
        uint32_t pk[kKeys / 2];
#pragma unroll
        for (int e = 0; e < kKeys / 2; ++e) {
          float e0, e1;
          f32x2_split(fma_f32x2(f32x2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])),
                                sc2x2, base2),
                      e0, e1);
          e0 = ex2(e0);
          e1 = ex2(e1);
          sum2[e & 1] = add_f32x2(sum2[e & 1], f32x2(e0, e1));
          pk[e] = pack_bf16(e0, e1);
        }
        tmem_st32(s_t, pk);
        float sa, sb;
        f32x2_split(add_f32x2(sum2[0], sum2[1]), sa, sb);
        l += sa + sb;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          // tensor memory is ordered by the fences around the arrival, which needs no more than
          // its default release
          if (PAIR)
            mbar_arrive_cluster(p_bar + 8 * (n & 1));
          else
            mbar_arrive(&p_full[i][n & 1]);
        }
        ++n;
      }
      if (n && ok)
        ok = __all_sync(0xffffffffu, wait_bar(&o_done[i], 0, abort_flag, p.status));
      if (ok) {
        tc_fence_after();
        const bool mine = r < p.G * p.TQ && t < rt.ntok;
        const int64_t tok = w.tok0 + i * span + rank * p.TQ + t;
        const int head = w.h * p.G + (r - t * p.G);
        const float vsc = p.v_scale ? __ldg(p.v_scale + w.h) : 1.f;
        const float inv = l == 0.f ? 0.f : vsc / l;
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          uint32_t y[32];
          if (n) {
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
          p.lse[tok * p.Hq + head] = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();  // no block leaves while the other may still signal it
  if (warp == 9) {
    tc_fence_after();
    if (PAIR)
      tmem_dealloc_pair(tmem, 512);
    else
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
  const int h = (int)blockIdx.y, k0 = (int)blockIdx.x * kPrefillKeys;
  pdl_wait_then_release();
  for (int b = (int)blockIdx.z; b < a.B; b += (int)gridDim.z) {
    const int len = min(max(__ldg(kv_len + b), 0), a.max_pages * a.page_size);
    const int n = __ldg(q_start + b + 1) - __ldg(q_start + b);
    if (n <= 0 || k0 >= len) continue;
    const int lo = a.window ? max(0, len - n - a.window + 1) : 0;
    if (k0 + kPrefillKeys <= lo && k0 >= a.n_sink) continue;
    const int64_t half = (int64_t)a.B * a.Hkv * lp * D;
    for (int x = (int)threadIdx.x; x < kPrefillKeys * CH; x += 256) {
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
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
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
  // the cache as [page][head][64-column half][token][64]
  const cuuint64_t dims[5] = {64, (cuuint64_t)p.page_size, (cuuint64_t)C::kHalves,
                              (cuuint64_t)a.Hkv, (cuuint64_t)p.num_pages};
  const cuuint64_t str[4] = {(cuuint64_t)token_stride * 2, 128, (cuuint64_t)head_stride * 2,
                             (cuuint64_t)page_stride * 2};
  // boxes of whole pages, or of the places of a tile that lie in one page
  const auto rows = [&](int most) {
    int r = 8;
    while (r < most && p.page_size % (2 * r) == 0) r *= 2;
    return r;
  };
  p.k_rows = rows(kKeys / C::kHalves);
  p.v_rows = rows(kKeys);
  const bool both_halves = C::kHalves > 1 && p.k_rows == kKeys / C::kHalves;
  const cuuint32_t box_k[5] = {64, (cuuint32_t)p.k_rows, both_halves ? 2u : 1u, 1, 1};
  const cuuint32_t box_v[5] = {64, (cuuint32_t)p.v_rows, 1, 1, 1};
  cudaError_t e = encode_bf16(&mk, k, 5, dims, str, box_k);
  if (e == cudaSuccess) e = encode_bf16(&mv, v, 5, dims, str, box_v);
  if (e != cudaSuccess) return e;
  auto kern = k_attn_prefill<D>;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
  if (e != cudaSuccess) return e;
  // units of two row tiles: the sum over sequences of ceil(n / unit) <= T / unit + B, and <= T
  const int64_t most = (int64_t)a.T / (2 * C::kBlocks * p.TQ) + a.B;
  const unsigned blocks =  // under 2^31 (host check)
      (unsigned)(most < a.T ? most : a.T) * (unsigned)a.Hkv * C::kBlocks;
  count_launches(1);
  if (C::kPair)
    return launch_pdl_cluster(kern, dim3(blocks), dim3(kThreads), C::kSmem, st, 2u, mq, mk, mv, p);
  return launch_pdl(kern, dim3(blocks), dim3(kThreads), C::kSmem, st, mq, mk, mv, p);
}

template <int D>
cudaError_t launch_unpack(const AttnDims& a, const void* k, const void* v, const int32_t* table,
                          const int32_t* kv_len, const int32_t* q_start, void* out, int64_t lp,
                          int* status, cudaStream_t st) {
  const dim3 grid((unsigned)(lp / kPrefillKeys), (unsigned)a.Hkv, (unsigned)(a.B < 65535 ? a.B : 65535));
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
  }
  return a.D == 64 ? launch<64>(a, q, k_cache, v_cache, p, ps, hs, ts, st)
                   : launch<128>(a, q, k_cache, v_cache, p, ps, hs, ts, st);
}

}  // namespace moe
