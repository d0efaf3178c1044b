// Attention of any number of new tokens per sequence over the paged cache (prompts, and chunks of
// prompts), on tcgen05 tensor cores.
//
//   s_ij = scale q_i.k_j over the places j that token i sees, o_i = sum_j softmax(s_i)_j v_j
//
// What bounds it: the tensor cores, 4 D flops per visible (query head, key) pair; next to them
// the exponentials, one per pair, and the chain of latencies from S to P of a row tile.
//
// Measured in bursts of 20 ms, 64 query heads of 128 on 8 key heads: 2048 tokens over 20011 places in
// E4M3, 784 us, 1.80 PFLOP/s of 1.89 that a library's matrix product reaches so; 8192 tokens, 656 us, 0.89
// of it; 8 ragged prompts of 65 to 3001 tokens, groups of 7, 321 us, 0.69 (one part in ten is the ends
// of units, when O drains to memory, one in twelve the masked halves of diagonal tiles); 37 tokens, 8.7
// us, latency. Back to back for a second the card's power limit takes the clock from 2070 MHz to 1870
// (1950 for the ragged prompts): 848 and 346 us. Heads of 64 do half the work in a tile's time: 32 heads,
// 8192 tokens, 340 us, 0.43, with a window of 1024, 117 us, 0.29: per tile of 64 places 600 cycles of exponentials (both row tiles' warps together)
// and 550 of loads, stores, votes and arrivals around them, against 512 of the tensor cores.
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
// memory. Heads of 64 are bound by the softmax before that and run on single blocks.
//
// Tensor memory: per row tile two buffers of 64 columns of scores S (fp32) and D columns of output
// O (fp32). The probabilities P (bf16) overwrite their S and are the A operand of the second
// product from there; K is K-major and V MN-major as TMA lays both down (rows of places, 128-byte
// swizzle).
//
// Warps: 0-3 softmax of row tile 0 (one row a thread), 4-7 of row tile 1, 8 TMA of Q and K, 10 of
// V, 9 and 11 the MMAs of row tiles 0 and 1 (in the pair's even block), one thread of each. One warp
// for all four was the bound: a tile takes the tensor cores about 1000 cycles, and each thread's
// waits, look-ups and issues 300 to 1000. The last warpgroup's registers go to the softmax warps.
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
constexpr int kRegs = 168;            // of a thread at launch: 384 * 168 = 128 * (200 + 200 + 104)
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kNoMax = -3e38f;     // the maximum of no scores: finite, so that -inf - it is -inf

struct Cut;

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
  float* parts;       // split units: unnormalised outputs, and their running maxima and sums
  float2* part_ml;
  Cut* cuts;   // where each run begins, for the join
  int min_split;      // key tiles of the shortest unit that is cut
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
  static constexpr int kSlots = 8;                          // of K, and of V
  static constexpr uint32_t kStage = 32 * 128;              // a softmax warp's rows, 128 bytes of each
  static constexpr uint32_t kQBytes = 2 * kQTile;
  static constexpr uint32_t kSmem = kQBytes + 2 * kSlots * kSlot + 8 * kStage + 1024;
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
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// ---- the split of the work ----------------------------------------------------------------------
// A unit is two row tiles of one sequence and key head (in a pair, two of 256 rows): `unit_tok`
// tokens. All units in a row (sequence, key head, tokens ascending), each weighed by the places
// that its last token sees plus kUnitCost for its start and end, are cut into equal runs, one per
// block (pair) of a grid that fills the SMs, but of a tile at least. A run may begin and end inside a
// unit, whose parts k_attn_prefill_join then joins; cuts that would leave less than kMinPart key tiles
// on a side, or that fall into a unit of less than `min_split`, move to the unit's nearer end. A cut
// costs about 10 us in all, a tile 0.7 us: where there are units enough for every run, units of less than 48
// tiles stay whole, else of less than 16. Cut against whole, us: 1024 units of 18 tiles 126 against
// 117; 8 prompts of 1024 tokens (512 units of up to 17) 149 against 135; 256 units of up to 345, 779
// against 897. With few units: 16 tokens over 8192 places 32 against 71, over 2048 23 against 24;
// of up to 9 tiles, 512 tokens, 26 against 19. A unit's start and end weighed as 4, 6, 8 tiles, us: 8
// ragged prompts 321, 326, 342; one of 2048 tokens 66, 69, 71; one over 20011 places 779, 788, 780.
constexpr int kUnitCost = 4 * kKeys, kMinPart = 4, kSplitFew = 16, kSplitMany = 48;

// n / d of non-negative numbers: a 32-bit division where both fit
__device__ __forceinline__ int64_t div_s(int64_t n, int64_t d) {
  return ((n | d) >> 32) == 0 ? (int64_t)((uint32_t)n / (uint32_t)d) : n / d;
}

// One sequence's new tokens.
struct Seq {
  int q0, nq, len;  // first row of q, new tokens, kv_len
};

__device__ __forceinline__ Seq seq_of(const PrefillParams& p, int b) {
  Seq s;
  s.q0 = min(max(__ldcg(p.q_start + b), 0), p.T);
  s.nq = min(max(__ldcg(p.q_start + b + 1), s.q0), p.T) - s.q0;
  s.len = __ldcg(p.kv_len + b);
  return s;
}

// Weight of a sequence's first k units (of one key head): kUnitCost each, and the places up to a
// unit's end, none before place 0 and `cap` at most.
__device__ __forceinline__ int64_t weight(const PrefillParams& p, const Seq& s, int unit_tok,
                                          int k) {
  const int64_t pos0 = (int64_t)min(max(s.len, 0), p.max_len) - s.nq;
  const int64_t cap = (int64_t)p.window + unit_tok + p.n_sink;
  // unit j ends at pos0 + (j + 1) unit_tok: below 0 for j < a, at most cap for j < c
  const int64_t a = pos0 < 0 ? min((int64_t)k, div_s(-pos0, unit_tok)) : 0;
  int64_t c = k;
  if (p.window) c = max(a, min(c, cap > pos0 ? div_s(cap - pos0, unit_tok) : 0));
  return (int64_t)kUnitCost * k + (c - a) * pos0 + unit_tok * (c * (c + 1) - a * (a + 1)) / 2 +
         cap * (k - c);
}

// A unit: sequence, key head, number among the sequence's units.
struct Unit {
  int b, h, u;
  Seq s;
};

// A place in the row of units: a unit, and the first step in it.
struct Cut {
  Unit at;
  int step;
  int64_t x0;          // where the unit begins in the row
  int64_t each, more;  // weight of a run; the first `more` have one more
};

// What a unit's roles need.
struct Work {
  int h;
  int tok0, ntok;     // first row of q, tokens (over all row tiles)
  int pos0;           // place of the first token
  int len;            // kv_len
  int sink_tiles;     // key tiles 0 .. that hold sinks
  int lo, n;          // first tile of the window; steps, sinks that lie before lo included
  int lead;           // of these, sink tiles before lo
};

__device__ __forceinline__ Work work_of(const PrefillParams& p, const Unit& t, int unit_tok) {
  Work w;
  const int at = t.u * unit_tok;
  w.h = t.h;
  w.tok0 = t.s.q0 + at;
  w.ntok = min(unit_tok, t.s.nq - at);
  w.len = min(max(t.s.len, 0), p.max_len);
  w.pos0 = w.len - t.s.nq + at;
  const int last = w.pos0 + w.ntok - 1;
  const int end = last >= 0 ? last / kKeys + 1 : 0;  // tiles up to the last token
  w.lo = p.window ? min(end, max(0, w.pos0 - p.window + 1) / kKeys) : 0;
  w.sink_tiles = (p.n_sink + kKeys - 1) / kKeys;
  w.lead = min(w.sink_tiles, w.lo);
  w.n = w.lead + end - w.lo;
  return w;
}

// key tile of step j
__device__ __forceinline__ int key_tile(const Work& w, int j) {
  return j < w.lead ? j : w.lo + j - w.lead;
}

// the next unit; false past the last
__device__ __forceinline__ bool next_unit(const PrefillParams& p, int unit_tok, Unit& t) {
  if ((t.u + 1) * unit_tok < t.s.nq) {
    ++t.u;
    return true;
  }
  t.u = 0;
  if (++t.h < p.Hkv) return true;
  t.h = 0;
  while (++t.b < p.B) {
    t.s = seq_of(p, t.b);
    if (t.s.nq > 0) return true;
  }
  return false;
}

// Where run c of `runs` begins, found by a warp.
__device__ __forceinline__ Cut find_cut(const PrefillParams& p, int unit_tok, int c, int runs) {
  const int lane = (int)threadIdx.x & 31;
  const auto all_of = [&](const Seq& s) {
    return s.nq > 0 ? weight(p, s, unit_tok, (s.nq + unit_tok - 1) / unit_tok) : 0;
  };
  int64_t total = 0;
  Seq held{0, 0, 0};  // of sequence `lane`
  for (int b = lane; b < p.B; b += 32) {
    const Seq s = seq_of(p, b);
    if (s.nq > 0 && (s.len < 0 || s.len > p.max_len))
      record_error(p.status, MOE_ERR_DEVICE_BOUNDS);
    if (b < 32) held = s;
    total += all_of(s);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  total *= p.Hkv;
  // A run is a tile at least, so that no two cuts of a unit fall on the same step: the join takes a
  // part from every run between a unit's first and last cut. Runs past the end take nothing.
  const int64_t shared = max(total, (int64_t)runs * kKeys);
  const int64_t each = div_s(shared, runs), more = shared - each * runs;
  int64_t x = c * each + min((int64_t)c, more);
  const int64_t here = x;
  Cut cut;
  cut.x0 = 0;
  cut.each = each;
  cut.more = more;
  cut.at.b = p.B;
  cut.at.h = cut.at.u = cut.step = 0;
  cut.at.s = Seq{0, 0, 0};
  if (x >= total) return cut;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    Seq s = held;
    if (b0) s = b0 + lane < p.B ? seq_of(p, b0 + lane) : Seq{0, 0, 0};
    const int64_t mine = all_of(s) * p.Hkv;
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    const int64_t all = __shfl_sync(0xffffffffu, incl, 31);
    if (x < all) {
      const int at = __popc(__ballot_sync(0xffffffffu, incl <= x));
      x -= __shfl_sync(0xffffffffu, incl - mine, at);
      cut.at.b = b0 + at;
      cut.at.s.q0 = __shfl_sync(0xffffffffu, s.q0, at);
      cut.at.s.nq = __shfl_sync(0xffffffffu, s.nq, at);
      cut.at.s.len = __shfl_sync(0xffffffffu, s.len, at);
      break;
    }
    x -= all;
  }
  const int64_t of_head = all_of(cut.at.s);
  cut.at.h = (int)div_s(x, of_head);
  x -= cut.at.h * of_head;
  // the last unit that begins by x, 32 probes a round
  int lo = 0, among = (cut.at.s.nq + unit_tok - 1) / unit_tok;
  while (among > 1) {
    const int gap = (among + 31) / 32, k = lane * gap;
    const bool by = k < among && weight(p, cut.at.s, unit_tok, lo + k) <= x;
    const int last = __popc(__ballot_sync(0xffffffffu, by)) - 1;
    lo += last * gap;
    among = min(gap, among - last * gap);
  }
  cut.at.u = lo;
  x -= weight(p, cut.at.s, unit_tok, lo);
  cut.x0 = here - x;
  const int n = work_of(p, cut.at, unit_tok).n;
  int step = x <= kUnitCost ? 0 : (int)min((int64_t)n, (x - kUnitCost) / kKeys);
  if (n < p.min_split) step = 2 * step < n ? 0 : n;
  if (step < kMinPart) step = 0;
  if (step > n - kMinPart && x > 0) step = n;
  cut.step = step;
  if (step == n && x > 0) {  // the next unit's beginning
    cut.step = 0;
    if (!next_unit(p, unit_tok, cut.at)) cut.at.b = p.B;
  }
  return cut;
}

__device__ __forceinline__ bool same_unit(const Unit& x, const Unit& y) {
  return x.b == y.b && x.h == y.h && x.u == y.u;
}

// Tokens [first, first + span) of a unit: the places p0 .. p1 of the first and the last of them,
// and, of the unit's steps s0 .. s1 - 1, those in [a0, a1) and [b0, b1) whose key tiles any of
// them sees; `last` is the last of these, or -1.
struct RowTile {
  int p0, p1, ntok;
  int a0, a1, b0, b1, last;
};

__device__ __forceinline__ RowTile row_tile(const PrefillParams& p, const Work& w, int first,
                                            int span, int s0, int s1) {
  RowTile r;
  r.ntok = min(span, w.ntok - first);
  r.p0 = w.pos0 + first;
  r.p1 = r.p0 + r.ntok - 1;
  const bool any = r.ntok > 0 && r.p1 >= 0;
  const int lo = p.window ? max(0, r.p0 - p.window + 1) / kKeys : 0;
  const int skip = w.lo - w.lead;  // tiles between the sinks' and the window's
  const int to = any ? r.p1 / kKeys + 1 - skip : 0;
  // sink tiles past the window's first are among its steps
  const int sink = min(to, w.sink_tiles > w.lo ? w.sink_tiles - skip : w.lead);
  r.a0 = s0;
  r.a1 = max(s0, min(sink, s1));
  r.b0 = max(r.a1, max(lo - skip, s0));
  r.b1 = max(r.b0, min(to, s1));
  r.last = r.b1 > r.b0 ? r.b1 - 1 : r.a1 > r.a0 ? r.a1 - 1 : -1;
  return r;
}

__device__ __forceinline__ bool sees(const RowTile& r, int j) {
  return (j >= r.a0 && j < r.a1) || (j >= r.b0 && j < r.b1);
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

// a mask of the columns 0 .. n - 1 of a tile
__device__ __forceinline__ uint64_t below(int n) {
  return n <= 0 ? 0 : n >= 64 ? ~0ull : (1ull << n) - 1;
}

// Row of the workspace's parts where row 0 of part `which` of run c lies: row tile i of block `rank`.
template <class C>
__device__ __forceinline__ int64_t part_row(int c, int which, int i, int rank) {
  return ((((int64_t)c * 2 + which) * C::kBlocks + rank) * 2 + i) * kRows;
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
  uint8_t* stage = ring + 2 * C::kSlots * C::kSlot;
  // Phases: q_full, q_empty once a unit; tail_full once a unit that has a tail; o_done, o_free once a
  // unit of which the row tile sees anything; the others once a tile.
  // q_full, full, p_full and o_free are waited on in the pair's even block.
  __shared__ uint64_t q_full, q_empty, s_full[2][2], p_full[2][2], o_full[2][2], o_done[2], o_free[2],
      tail_full, full[2][C::kSlots], empty[2][C::kSlots];  // of K, of V
  __shared__ uint32_t tmem_holder;
  __shared__ int abort_flag_s;
  __shared__ Cut cut_s[2];
  volatile int* abort_flag = &abort_flag_s;
  const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31;
  const int rank = PAIR ? (int)cluster_ctarank() : 0;

  if (threadIdx.x == 0) {
    mbar_init(&q_full, 1);
    mbar_init(&q_empty, 2);                           // both row tiles' MMAs have read it
    for (int i = 0; i < 2; ++i) {
      mbar_init(&o_done[i], 1);                       // the last PV
      mbar_init(&o_free[i], 4 * C::kBlocks);          // the row tile's warps
      for (int b = 0; b < 2; ++b) {
        mbar_init(&s_full[i][b], 1);
        mbar_init(&o_full[i][b], 1);                  // a phase for every second PV
        mbar_init(&p_full[i][b], 4 * C::kBlocks);
      }
    }
    mbar_init(&tail_full, 1);
    for (int s = 0; s < C::kSlots; ++s) {
      for (int kv = 0; kv < 2; ++kv) {
        mbar_init(&full[kv][s], kv ? C::kBlocks : 1);  // V: every block, for the tails' sake
        mbar_init(&empty[kv][s], 2);                  // both row tiles' MMAs have read it
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

  // ---- this run: from the first cut to the second ----
  const int span = p.TQ * C::kBlocks;  // tokens of a row tile of the unit
  const int unit_tok = 2 * span;
  const int run = (int)blockIdx.x / C::kBlocks, runs = (int)gridDim.x / C::kBlocks;
  if (warp == 8 || warp == 10) {
    const Cut c = find_cut(p, unit_tok, run + (warp == 10), runs);
    if (lane == 0) {
      cut_s[warp == 10] = c;
      if (p.cuts && warp == 8 && rank == 0) p.cuts[run] = c;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();  // both blocks' barriers are initialised
  tc_fence_after();
  const uint32_t tmem = tmem_holder;
  const Cut stop = cut_s[1];
  // the run's parts: a unit and its steps [s0, s1) at a time
  struct Part {
    Unit t;
    Work w;
    int s0, s1;
    bool tail;  // places past kv_len share the last tile (of a cache read in place) with earlier ones
  };
  const auto fill = [&](Part& x, int s0) {
    x.w = work_of(p, x.t, unit_tok);
    x.s0 = s0;
    x.s1 = same_unit(x.t, stop.at) ? stop.step : x.w.n;
    x.tail = p.block_table && x.s1 > s0 && x.s1 == x.w.n &&
             (key_tile(x.w, x.w.n - 1) + 1) * kKeys > x.w.len;
  };
  const auto first_part = [&](Part& x) {
    x.t = cut_s[0].at;
    if (x.t.b >= p.B || (same_unit(x.t, stop.at) && stop.step <= cut_s[0].step)) return false;
    fill(x, cut_s[0].step);
    return true;
  };
  const auto next_part = [&](Part& x) {
    if (same_unit(x.t, stop.at) || !next_unit(p, unit_tok, x.t)) return false;
    if (same_unit(x.t, stop.at) && stop.step == 0) return false;
    fill(x, 0);
    return true;
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp == 8 || warp == 10) {
      // ---------------- TMA: warp 8 Q and K, warp 10 V (one thread each) ----------------
      const int kv = warp == 8 ? 0 : 1;
      const uint32_t ring_kv = smem_u32(ring) + kv * (C::kSlots * C::kSlot);
      // A tile's boxes: rows box * rows .. of this block's part. K of a pair: its 32 places, both
      // 64-column halves (in one box if that takes all 32, else box by box); V of a pair: all 64
      // places of its half; else all 64 places.
      constexpr int kKRows = kKeys / C::kHalves;
      const int rows = kv ? p.v_rows : p.k_rows;
      const int part = kv ? kKeys : kKRows;                 // places of the block's part
      const int first = kv ? 0 : rank * kKRows;             // its first place of a tile
      const int half = kv && PAIR ? rank : 0;
      const CUtensorMap* map = kv ? &tm_v : &tm_k;
      const uint32_t full_bar =
          PAIR ? mapa_shared(smem_u32(&full[kv][0]), 0) : smem_u32(&full[kv][0]);
      int slot = 0;
      uint32_t phase = 0, units = 0, tails = 0;
      int64_t issued = 0;
      bool ok = true;
      Part x;
      for (bool more = first_part(x); more; more = next_part(x)) {
        const Work& w = x.w;
        if (elect_one()) {
          if (kv == 0) {
            const uint32_t bytes = C::kHalves * (uint32_t)(p.G * p.TQ) * 128;
            ok = wait_bar(&q_empty, (units & 1) ^ 1u, abort_flag, p.status);
            if (ok) {
              const int tiles = w.ntok > span ? 2 : 1;
              if (rank == 0) mbar_arrive_expect_tx(&q_full, C::kBlocks * tiles * bytes);
              const uint32_t bar = PAIR ? mapa_shared(smem_u32(&q_full), 0) : smem_u32(&q_full);
              for (int i = 0; i < tiles; ++i)
                for (int hf = 0; hf < C::kHalves; ++hf)
                  tma_load_3d<PAIR>(smem_u32(q_s) + i * C::kQTile + hf * C::kHalfBytes, &tm_q, bar,
                                    hf * 64, w.h * p.G, w.tok0 + i * span + rank * p.TQ);
            }
          }
          const int end = min(w.len, w.pos0 + w.ntok);          // places any row sees
          const int lo = p.window ? max(0, w.pos0 - p.window + 1) : 0;
          const int32_t* table = p.block_table + (int64_t)x.t.b * p.max_pages;
          // the last V tile is completed in shared memory if it ends past kv_len
          const int n = x.s1 - (kv == 1 && x.tail ? 1 : 0);
          const auto tiles = [&](auto row_boxes, auto halves) {
            constexpr int NR = decltype(row_boxes)::value;
            constexpr bool split = decltype(halves)::value;  // halves of K in boxes of their own
            // pages of a tile's boxes and their rows there, looked up a step before they are used;
            // bit b of `in`: some row of the unit sees box b (others come from beyond the map: zeros)
            int page[NR], row[NR];
            uint32_t in = 0;
            const auto look_up = [&](int j) {
              const int key0 = key_tile(w, j) * kKeys + first;
              in = 0;
#pragma unroll
              for (int b = 0; b < NR; ++b) {
                const int key = key0 + b * rows;
                page[b] = p.num_pages;
                row[b] = 0;
                if (key < end && (key + rows > lo || key < p.n_sink)) {
                  in |= 1u << b;
                  page[b] = x.t.b;
                  row[b] = key;
                  if (p.block_table) {
                    const int pg = (int)div_fast((uint32_t)key, p.page_div);
                    page[b] = __ldg(table + pg);
                    row[b] = key - pg * p.page_size;
                  }
                }
              }
            };
            const auto load = [&](uint32_t dst, uint32_t bar, auto pair) {
              constexpr bool P = decltype(pair)::value;
              uint32_t out = 0;
#pragma unroll
              for (int b = 0; b < NR; ++b) {
                const uint32_t pg = min((uint32_t)page[b], (uint32_t)p.num_pages);
                if (pg == (uint32_t)p.num_pages) out |= 1u << b;
                const uint32_t at = dst + b * rows * 128;
                tma_load_5d<P>(at, map, bar, 0, row[b], half, w.h, pg);
                if (split) tma_load_5d<P>(at + C::kKHalf, map, bar, 0, row[b], 1, w.h, pg);
              }
              if (out & in) record_error(p.status, MOE_ERR_DEVICE_BOUNDS);
            };
            if (x.s0 < x.s1) look_up(x.s0);
            for (int j = x.s0; ok && j < x.s1; ++j) {
              ok = wait_bar(&empty[kv][slot], phase ^ 1u, abort_flag, p.status);
              if (!ok) break;
              const uint32_t dst = ring_kv + slot * C::kSlot;
              if (j < n) {
                if (rank == 0)
                  mbar_arrive_expect_tx(&full[kv][slot], C::kBlocks * C::kSlot);
                else if (kv == 1)
                  mbar_arrive_cluster(full_bar + 8 * slot);
                load(dst, full_bar + 8 * slot, std::integral_constant<bool, PAIR>());
              } else {
                mbar_arrive_expect_tx(&tail_full, C::kSlot);
                load(dst, smem_u32(&tail_full), std::integral_constant<bool, false>());
              }
              if (j + 1 < x.s1) look_up(j + 1);
              ++issued;
              if (++slot == C::kSlots) { slot = 0; phase ^= 1u; }
            }
          };
          using std::integral_constant;
          if (part == rows)
            tiles(integral_constant<int, 1>(), std::false_type());
          else if (PAIR && kv == 0)
            tiles(integral_constant<int, 2>(), std::true_type());
          else if (part == 2 * rows)
            tiles(integral_constant<int, 2>(), std::false_type());
          else
            tiles(integral_constant<int, 4>(), std::false_type());
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ++units;
        if (kv == 1 && x.tail) {
          // the places of the last V tile past kv_len: zeros; only then has the tile arrived
          ok = wait_bar(&tail_full, tails & 1, abort_flag, p.status);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          ++tails;
          const int lead = __ffs(__ballot_sync(0xffffffffu, issued > 0)) - 1;
          const int at = (__shfl_sync(0xffffffffu, slot, lead) + C::kSlots - 1) % C::kSlots;
          const int r0 = w.len - key_tile(w, w.n - 1) * kKeys;
          uint8_t* vt = ring + (C::kSlots + at) * C::kSlot;
          for (int e = lane; e < (kKeys - r0) * 8; e += 32)
            *reinterpret_cast<uint4*>(vt + (r0 + e / 8) * 128 + (e & 7) * 16) =
                make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (PAIR)
              mbar_arrive_release_cluster(full_bar + 8 * at);
            else
              mbar_arrive(&full[1][at]);
          }
        }
      }
      // every load issued has landed before the block may exit (in pairs the even block's barriers
      // count both blocks' bytes)
      if (rank == 0) {
        for (int s = 0; s < C::kSlots; ++s)
          if (s < issued) drain_bar(&full[kv][s], s < slot ? phase : phase ^ 1u, p.status);
        if (kv == 0 && units) drain_bar(&q_full, (units - 1) & 1, p.status);
      }
      // and so have the arrivals that hand slots and queries back
      if (__all_sync(0xffffffffu, ok)) {
        for (int s = 0; s < C::kSlots; ++s)
          if (s < issued) drain_bar(&empty[kv][s], s < slot ? phase : phase ^ 1u, p.status);
        if (kv == 0 && units) drain_bar(&q_empty, (units - 1) & 1, p.status);
      }
    } else if ((warp == 9 || warp == 11) && rank == 0) {
      // ------------ MMA: warp 9 row tile 0, warp 11 row tile 1 (one thread each) ------------
      const int i = warp == 9 ? 0 : 1;
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
        uint32_t n_qk = 0, n_pv = 0;  // products issued: the buffer and phase of the next
        int ks = 0, vs = 0;           // slots of the next K and V tile
        uint32_t kp = 0, vp = 0;
        uint32_t units = 0, seen = 0;
        bool ok = true;
        RowTile rt;
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
        Part x;
        for (bool more = first_part(x); ok && more; more = next_part(x)) {
          rt = row_tile(p, x.w, i * span, span, x.s0, x.s1);
          ok = wait_bar(&q_full, units & 1, abort_flag, p.status);
          if (!ok) break;
          for (int j = x.s0; ok && j < min(x.s0 + 2, x.s1); ++j) {
            ok = wait_bar(&full[0][ks], kp, abort_flag, p.status);
            if (!ok) break;
            tc_fence_after();
            qk(j);
            free_k();
          }
          if (x.s1 - x.s0 <= 2) commit(&q_empty);
          bool begun = false;
          for (int j = x.s0; ok && j < x.s1; ++j) {
            const bool ahead = j + 2 < x.s1, pv = sees(rt, j);
            // Most often everything is there: the tests of V, K and P travel together, where one
            // wait after the other would take 120 cycles each.
            const bool v_here = mbar_test_wait(&full[1][vs], vp);
            const bool k_here = mbar_test_wait(&full[0][ks], kp) | !ahead;
            const bool p_here = mbar_test_wait(&p_full[i][n_pv & 1], (n_pv >> 1) & 1) | !pv;
            if (!(v_here & k_here & p_here) || (pv && !begun) || (x.tail && j + 1 == x.s1)) {
              // the operands first: once P is there, nothing else holds up the products
              ok = x.tail && j + 1 == x.s1 ? wait_bar_pair(&full[1][vs], vp, abort_flag, p.status)
                                           : wait_bar(&full[1][vs], vp, abort_flag, p.status);
              if (ok && ahead) ok = wait_bar(&full[0][ks], kp, abort_flag, p.status);
              if (ok && pv && !begun)
                ok = wait_bar(&o_free[i], (seen & 1) ^ 1u, abort_flag, p.status);
              if (ok && pv)
                ok = wait_bar(&p_full[i][n_pv & 1], (n_pv >> 1) & 1, abort_flag, p.status);
              if (!ok) break;
            }
            tc_fence_after();
            if (pv) {  // O += P V(j)
              const uint64_t dv = dv0 + (uint64_t)(vs * (int)(C::kSlot >> 4));
              const uint32_t pa = s_t + (n_pv & 1) * kKeys;
#pragma unroll
              for (int kk = 0; kk < kKeys / 16; ++kk) {
                const uint64_t at = dv + (uint64_t)(kk * (2048 >> 4));
                const uint32_t acc = (begun || kk) ? 1u : 0u;
                if (PAIR)
                  mma_ts_pair(o_t, pa + 8 * kk, at, idesc_o, acc);
                else
                  mma_ts(o_t, pa + 8 * kk, at, idesc_o, acc);
              }
              ++n_pv;
              begun = true;
            }
            if (ahead) qk(j + 2);
            if (pv) commit(&o_full[i][(n_pv & 1) ^ 1]);
            if (j == rt.last) commit(&o_done[i]);
            commit(&empty[1][vs]);
            if (++vs == C::kSlots) { vs = 0; vp ^= 1u; }
            if (ahead) {
              free_k();
              if (j + 3 == x.s1) commit(&q_empty);  // the unit's queries are read
            }
          }
          ++units;
          if (begun) ++seen;
        }
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    // ---------------- softmax and epilogue ----------------
    const int i = warp >> 2;
    const int r = (warp & 3) * 32 + lane;                 // row of the tile
    const int t = (int)div_fast((uint32_t)r, p.g_div);    // its token
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t o_t = lanes + C::kTmemO + i * D;
    const uint32_t p_bar = PAIR ? mapa_shared(smem_u32(&p_full[i][0]), 0) : 0;
    const uint32_t o_bar = PAIR ? mapa_shared(smem_u32(&o_free[i]), 0) : 0;
    uint32_t n = 0, seen = 0;  // tiles done; units seen anything of
    bool ok = true;
    Part x;
    for (bool more = first_part(x); more; more = next_part(x)) {
      const Work& w = x.w;
      // the row tile over all blocks
      const RowTile both = row_tile(p, w, i * span, span, x.s0, x.s1);
      const int p0 = w.pos0 + i * span + rank * p.TQ;                 // of this block's rows
      const int ntok = min(p.TQ, w.ntok - i * span - rank * p.TQ);
      const int pos = p0 + t;
      const float sc2 = p.scale * kLog2e * (p.k_scale ? __ldg(p.k_scale + w.h) : 1.f);
      // key tiles whose every place every row sees: the first ones to, and of these those from (or
      // of sinks alone)
      const int plain_to = (p0 + 1) / kKeys;
      const int plain_from = p.window ? max(0, p0 + ntok - 1 - p.window + kKeys) / kKeys : 0;
      const int plain_sink = p.n_sink / kKeys;
      // the running maximum and sum, the maximum as a base-2 exponent
      float m = kNoMax, l = 0.f;
      bool begun = false;
      for (int j = both.a1 > both.a0 ? both.a0 : both.b0; j < both.b1 || j < both.a1;
           j = j + 1 == both.a1 ? both.b0 : j + 1) {
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
          // columns up to `hi` are seen, but for those up to `lo` that are not before `sk`
          const int hi = pos - k0, lo = p.window ? hi - p.window : -1, sk = p.n_sink - k0;
          const uint64_t seen = below(hi + 1) & ~(below(lo + 1) & ~below(sk));
#pragma unroll
          for (int c = 0; c < kKeys; ++c)
            if (!(seen >> c & 1)) s[c] = 0xFF800000u;
          // the load's maximum is that of every column: good enough unless it would raise m
          if (__any_sync(0xffffffffu, fmaxf(mx2[0], mx2[1]) * sc2 > m + 8.f)) {
            mx2[0] = mx2[1] = -INFINITY;
#pragma unroll
            for (int c = 0; c < kKeys; ++c) mx2[c & 1] = fmaxf(mx2[c & 1], __uint_as_float(s[c]));
          }
        }
        const float mx = fmaxf(mx2[0], mx2[1]) * sc2;
        // raise the running maximum only where it is exceeded by 2^8 (or has no value yet)
        const bool raise = mx > m + 8.f;
        if (__any_sync(0xffffffffu, raise)) {
          const float f = raise ? ex2(m - mx) : 1.f;
          if (raise) m = mx;
          l *= f;
          if (begun) {
            // PV of the tile before. When S(n) is there, the arrival of PV(n-2), committed right after
            // it, may still be on its way, so barriers alternate: in one for all, the phase of PV(n-1)
            // has the parity of PV(n-3)'s and would pass for done.
            ok = wait_bar(&o_full[i][(n - 1) & 1], ((n - 1) >> 1) & 1, abort_flag, p.status);
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
        begun = true;
        ++n;
      }
      if (!ok) break;
      if (begun) {
        ok = wait_bar(&o_done[i], seen & 1, abort_flag, p.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ++seen;
        tc_fence_after();
      }
      // O through shared memory, 128 bytes of a row at a time, so that a store writes whole lines:
      // of 32 rows a thread each, every store would touch 32.
      const bool whole = x.s0 == 0 && x.s1 == w.n;
      const int rows_in = min(p.G * p.TQ, p.G * ntok);    // rows of this block's row tile
      const int64_t part0 = part_row<C>(run, x.s0 > 0 ? 0 : 1, i, rank);
      const int64_t tok0 = w.tok0 + i * span + rank * p.TQ;
      uint8_t* st = stage + warp * C::kStage;
      const float vsc = p.v_scale ? __ldg(p.v_scale + w.h) : 1.f;
      const float inv = l == 0.f ? 0.f : vsc / l;
      const auto put = [&](int chunk, uint32_t z0, uint32_t z1, uint32_t z2, uint32_t z3) {
        *reinterpret_cast<uint4*>(st + lane * 128 + ((chunk ^ lane) & 7) * 16) =
            make_uint4(z0, z1, z2, z3);
      };
      // the lane's rows when the warp writes: 8 lanes to a row, rows 4e + lane / 8
      const int row0 = (warp & 3) * 32 + (lane >> 3), chunk = lane & 7;
      const auto take = [&](int e) {
        return *reinterpret_cast<const uint4*>(st + (4 * e + (lane >> 3)) * 128 +
                                               ((chunk ^ (4 * e + (lane >> 3))) & 7) * 16);
      };
      if (whole) {
        uint16_t* to[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int row = row0 + 4 * e, tk = (int)div_fast((uint32_t)row, p.g_div);
          to[e] = p.o + (tok0 + tk) * p.o_stride + (w.h * p.G + row - tk * p.G) * D + chunk * 8;
        }
        const uint64_t inv2 = f32x2(inv, inv);
#pragma unroll
        for (int c = 0; c < D; c += 64) {
          uint32_t y[64];
          if (begun) {
            tmem_ld32(o_t + c, y);
            tmem_ld32(o_t + c + 32, y + 32);
            tmem_ld_wait32(y);
            tmem_ld_wait32(y + 32);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            uint32_t z[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float a, b;
              f32x2_split(mul_f32x2(f32x2(__uint_as_float(y[8 * e + 2 * k]),
                                          __uint_as_float(y[8 * e + 2 * k + 1])), inv2), a, b);
              z[k] = inv == 0.f ? 0u : pack_bf16(a, b);
            }
            put(e, z[0], z[1], z[2], z[3]);
          }
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (row0 + 4 * e < rows_in) *reinterpret_cast<uint4*>(to[e] + c) = take(e);
          __syncwarp();
        }
      } else if (begun) {
        float* to = p.parts + (part0 + row0) * D + chunk * 4;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t y[32];
          tmem_ld32(o_t + c, y);
          tmem_ld_wait32(y);
#pragma unroll
          for (int e = 0; e < 8; ++e) put(e, y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (row0 + 4 * e < rows_in) *reinterpret_cast<uint4*>(to + 4 * e * D + c) = take(e);
          __syncwarp();
        }
      }
      if (r < rows_in) {
        if (!whole)  // the run's first part if the unit began before it, else its second
          p.part_ml[part0 + r] = make_float2(m, l);
        else if (p.lse)
          p.lse[(tok0 + t) * p.Hq + w.h * p.G + (r - t * p.G)] =
              l == 0.f ? -INFINITY : m * kLn2 + logf(l);
      }
      if (begun) {  // the next unit's products may overwrite O
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (PAIR)
            mbar_arrive_cluster(o_bar);
          else
            mbar_arrive(&o_free[i]);
        }
      }
    }
    // The last products' arrivals, which no tile follows that could wait for them to raise the maximum:
    // here before the block may leave.
    if (ok && n > 1) drain_bar(&o_full[i][n & 1], ((n - 2) >> 1) & 1, p.status);
    if (ok && n) drain_bar(&o_full[i][(n - 1) & 1], ((n - 1) >> 1) & 1, p.status);
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

// Joins the parts of the units that runs cut: kJoin blocks look at the cut between two runs, and the
// cuts of one unit share its (row, eight columns) tasks, in the parts' order. Bound by reading the parts:
// 75 cuts of units of 512 rows of 128, 39 MB, 16 us.
constexpr int kJoin = 16;

template <int D>
__global__ void __launch_bounds__(256) k_attn_prefill_join(const PrefillParams p) {
  using C = Cfg<D>;
  const int unit_tok = 2 * p.TQ * C::kBlocks;
  const int c = (int)blockIdx.x / kJoin + 1, mine = (int)blockIdx.x % kJoin;
  pdl_wait_then_release();
  const Cut cut = p.cuts[c];
  if (cut.step == 0) return;
  // The cuts inside the unit are those whose step is kMinPart .. n - kMinPart: from y to z - 1 in
  // the row. Run c0 begins the unit, run c1 ends it.
  const auto run_of = [&](int64_t x) {  // the run that place x falls into
    const int64_t longer = cut.more * (cut.each + 1);
    return (int)(x < longer ? div_s(x, cut.each + 1) : cut.more + div_s(x - longer, cut.each));
  };
  const Work w = work_of(p, cut.at, unit_tok);
  const int64_t y = cut.x0 + kUnitCost + kMinPart * kKeys;
  const int64_t z = cut.x0 + kUnitCost + (int64_t)(w.n - kMinPart + 1) * kKeys;
  const int c0 = run_of(y - 1), c1 = run_of(z - 1);
  const int tasks = w.ntok * p.G * (D / 8);
  const int shares = (c1 - c0) * kJoin, share = (c - c0 - 1) * kJoin + mine;
  const int t0 = (int)((int64_t)tasks * share / shares);
  const int t1 = (int)((int64_t)tasks * (share + 1) / shares);
  const float vsc = p.v_scale ? __ldg(p.v_scale + w.h) : 1.f;
  for (int task = t0 + (int)threadIdx.x; task < t1; task += 256) {
    const int row = task / (D / 8), col = task % (D / 8) * 8;
    const int tk = (int)div_fast((uint32_t)row, p.g_div), g = row - tk * p.G;
    // token tk lies in row tile tk / span, block (tk % span) / TQ of the pair
    const int span = p.TQ * C::kBlocks, i = tk / span, rank = tk % span / p.TQ;
    const int r = (tk - i * span - rank * p.TQ) * p.G + g;
    float m = kNoMax, l = 0.f, sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int x = c0; x <= c1; ++x) {
      const int64_t at = part_row<C>(x, x == c0 ? 1 : 0, i, rank) + r;
      const float2 ml = __ldcg(p.part_ml + at);
      if (ml.y == 0.f) continue;  // the row saw nothing of the part
      const float4* src = reinterpret_cast<const float4*>(p.parts + at * D + col);
      const float4 lo = __ldcg(src), hi = __ldcg(src + 1);
      const float to = fmaxf(m, ml.x), f = ex2(m - to), e = ex2(ml.x - to);
      const float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
      l = l * f + ml.y * e;
#pragma unroll
      for (int k = 0; k < 8; ++k) sum[k] = fmaf(v[k], e, sum[k] * f);
      m = to;
    }
    const float inv = l == 0.f ? 0.f : vsc / l;
    const int64_t tok = w.tok0 + tk;
    const int head = w.h * p.G + g;
    uint32_t out[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) out[k] = pack_bf16(sum[2 * k] * inv, sum[2 * k + 1] * inv);
    *reinterpret_cast<uint4*>(p.o + tok * p.o_stride + (int64_t)head * D + col) =
        make_uint4(out[0], out[1], out[2], out[3]);
    if (p.lse && col == 0) p.lse[tok * p.Hq + head] = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
  }
}

// ---- caches that the tiles cannot read as they lie ---------------------------------------------
// Copies what this step's tokens see into rows in order: E4M3 codes become bf16 exactly (the
// scales stay outside), and places that no token sees but that share a tile with one are zeros.
// Bound by HBM: one read of the visible cache and one bf16 write, against 2 G n flops an element for
// n tokens a sequence. 22059 places of 8 key heads of 128, E4M3: 23 us, 0.87 of the copy rate. Its grid is
// as wide as the tables: 64 sequences of 1 to 64 places, 55 us with tables of 64 places, 574 with tables of 131072.
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

// key tiles of the longest unit that the shape allows
int64_t prefill_tiles_most(const AttnDims& a) {
  const int64_t places = (int64_t)a.max_pages * a.page_size;
  const int64_t seen = a.window ? (int64_t)a.window + a.n_sink + 2 * kRows * 2 : places;
  return (seen < places ? seen : places) / kKeys + 3;
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
    int r = 16;
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
  // the warps exchange registers: what they take has to be there at launch
  static const int regs = [&] {
    cudaFuncAttributes at{};
    return cudaFuncGetAttributes(&at, kern) == cudaSuccess ? at.numRegs : 0;
  }();
  if (regs != kRegs) return cudaErrorInvalidConfiguration;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
  if (e != cudaSuccess) return e;
  // Units: the sum over sequences of ceil(n / unit) <= T / unit + B, and <= T, for each key head. Where
  // no unit can be long enough to be cut, no more runs than units.
  const int64_t of_head = (int64_t)a.T / (2 * C::kBlocks * p.TQ) + a.B;
  const int64_t most = (of_head < a.T ? of_head : a.T) * a.Hkv;
  const int64_t full_units = (int64_t)(a.T / (2 * C::kBlocks * p.TQ)) * a.Hkv;  // about as many
  int runs = num_sms() / C::kBlocks;
  if (runs > kPrefillMaxCtas / C::kBlocks) runs = kPrefillMaxCtas / C::kBlocks;
  p.min_split = full_units >= runs ? kSplitMany : kSplitFew;
  const bool cuts = prefill_tiles_most(a) >= p.min_split;
  if (!cuts) p.cuts = nullptr;
  if (!cuts && runs > most) runs = (int)most;
  count_launches(cuts && runs > 1 ? 2 : 1);
  const dim3 grid((unsigned)(runs * C::kBlocks));
  e = C::kPair ? launch_pdl_cluster(kern, grid, dim3(kThreads), C::kSmem, st, 2u, mq, mk, mv, p)
               : launch_pdl(kern, grid, dim3(kThreads), C::kSmem, st, mq, mk, mv, p);
  if (e != cudaSuccess || !cuts || runs == 1) return e;
  return launch_pdl(k_attn_prefill_join<D>, dim3((unsigned)(runs - 1) * kJoin), dim3(256), 0, st,
                    p);
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
  p.parts = reinterpret_cast<float*>(ws + L.prefill_parts);
  p.part_ml = reinterpret_cast<float2*>(ws + L.prefill_ml);
  static_assert(sizeof(Cut) <= kPrefillCutBytes, "workspace");
  p.cuts = reinterpret_cast<Cut*>(ws + L.prefill_cuts);
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
