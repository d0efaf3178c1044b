// y = x w^T + bias + residual, both matrices in MXFP4, on block-scaled tcgen05.mma (kind::mxf4: 64 of
// K an instruction, one E8M0 scale per row and 32 of K, fp32 sums in TMEM).
//
// Up to 128 tokens, and more where few tiles have long rows: the weights are the M side (128 rows a tile), the tokens the N side, so that a single
// token streams each weight byte once at full tile width. A stage holds 256 of K: one 128-byte swizzle row of
// codes a matrix row and two 512-byte blocks of scales a side, which tcgen05.cp carries to TMEM ahead of the
// stage's four MMAs. Few tiles are split along K over the CTAs of a cluster; their fp32 sums meet in
// distributed shared memory, added in the order of K.
//
// What bounds it: HBM for large matrices (one token of 65536 x 7168: 38.6 us, 6.5 TB/s, 0.95 of the copy rate); for
// the usual ones the chain of a launch, the first loads, and the gathering of sums (3.4 us for 2304 x 1024)
// around the weights' 4 to 6 us (9216 x 7168: 7.2 us).
#include "mx_linear.cuh"
#include "mx_quant.cuh"

namespace moe {
namespace {

using namespace mxl;

constexpr int kQuantRows = 4;     // rows of 256 of K that a warp quantises in a block: 4 * 4 in all
constexpr int kQuantStages = 12;  // stages of x beside the ring: two blocks still share an SM
// Stages whose weights are on their way to L2 before the wait for the kernel ahead: 4 take one token of 9216 x
// 7168 from 8.0 to 7.3 us; 28, a long row whole, is more than L2 holds over all blocks (65536 x 7168: 50 us for 40).
constexpr int kAheadStages = 4;
constexpr int kLinThreads = 192;  // warps: 0 loads, 1 MMAs, 2..5 quantise x, then read the sums

// A ring of stages; x that the block quantises itself (QUANT) lies beside it whole.
template <int NT, int STAGES, bool QUANT>
struct LinSmem {
  static constexpr uint32_t kA = kBM * kRowBytes;
  static constexpr uint32_t kB = NT * kRowBytes;
  static constexpr uint32_t kTiles = STAGES * (kA + (QUANT ? 0 : kB));
  static constexpr uint32_t kScales = STAGES * (QUANT ? 1 : 2) * kSfBytes;
  static constexpr uint32_t kRing = kTiles + kScales;
  static constexpr uint32_t kX = QUANT ? kB + kSfBytes : 0;  // of a stage of x
  static constexpr uint32_t kPart = NT * kBM * 4;  // the sums, over the tiles once they are read
  static constexpr uint32_t kBars = 8 * (2 * STAGES + 2) + 16;
  static constexpr uint32_t total(int nx) { return kRing + nx * kX + kBars + 1024; }
  static constexpr uint32_t kSfCol = NT;  // scales: 2 x (8 columns of A, 8 of B)
  static constexpr uint32_t kCols = NT + 32 <= 64 ? 64 : NT + 32 <= 128 ? 128 : 256;
};

// The sums of S blocks for four rows of w, in the order of K; all S loads on their way at once.
template <int S>
__device__ __forceinline__ float4 gathered(uint32_t addr) {
  float4 a[S];
#pragma unroll
  for (int s = 0; s < S; ++s) a[s] = ld_cluster_f4(mapa_shared(addr, s));
#pragma unroll
  for (int s = 1; s < S; ++s) {
    a[0].x += a[s].x;
    a[0].y += a[s].y;
    a[0].z += a[s].z;
    a[0].w += a[s].w;
  }
  return a[0];
}

template <int NT, int STAGES, bool QUANT>
__global__ void __launch_bounds__(kLinThreads, 2)
    k_mx_linear(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                const LinParams p) {
  using S = LinSmem<NT, STAGES, QUANT>;
  static_assert(S::kPart <= S::kRing, "the sums fit over the ring");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const int nst = (p.chunks + 1) >> 1;
  const int rank = (int)(blockIdx.x % (unsigned)p.splits);
  const int k0 = (int)((long)nst * rank / p.splits), k1 = (int)((long)nst * (rank + 1) / p.splits);
  const int nx = QUANT ? (nst + p.splits - 1) / p.splits : 0;  // most stages of a block
  uint8_t* sm_b = smem + STAGES * S::kA;      // x's tiles: of the ring, or
  uint8_t* sm_x = smem + S::kRing;            // whole: tiles, then scales
  uint8_t* sm_sf = smem + S::kTiles;          // per stage: of w, of the ring's x
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::kRing + nx * S::kX);
  uint64_t* empty = full + STAGES;
  uint64_t* acc_full = empty + STAGES;
  uint64_t* x_full = acc_full + 1;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(x_full + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(x_full, 4);  // the quantising warps
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tm_w);
    if (!QUANT) prefetch_tmap(&tm_x);
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, S::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;

  const int tile = (int)(blockIdx.x / (unsigned)p.splits);
  const int mt = tile % p.mtiles, tt = tile / p.mtiles;
  const int row0 = mt * kBM, tok0 = tt * NT;
  const int ntok = min(NT, p.T - tok0);
  const int npad = (ntok + 15) & ~15;

  // Ahead of the wait for the kernel before: behind the call's own quantisation of x, which has itself
  // waited for everything before it, the first stages of the weights; else, as that kernel may still be
  // writing them, their way to L2 alone, where whatever it writes is written as well.
  const auto load_w = [&](int kb, uint32_t stage) {
    const uint32_t sf = (uint32_t)min(2, p.chunks - 2 * kb) * kMxTile;
    mbar_arrive_expect_tx(&full[stage], S::kA + sf + (QUANT ? 0u : S::kB + sf));
    tma_load_2d(smem + stage * S::kA, &tm_w, &full[stage], kb * (int)kRowBytes, row0,
                policy_evict_first());
    bulk_load(sm_sf + stage * (QUANT ? 1 : 2) * kSfBytes,
              p.w_scales + ((size_t)mt * p.chunks + 2 * kb) * kMxTile, sf, &full[stage]);
  };
  const int early = !QUANT && p.early ? min(STAGES, k1 - k0) : 0;
  if (warp == 0 && elect_one()) {
    for (int i = 0; i < early; ++i) load_w(k0 + i, (uint32_t)i);
    for (int kb = k0 + early; kb < min(k1, k0 + kAheadStages); ++kb)
      tma_prefetch_2d(&tm_w, kb * (int)kRowBytes, row0);
  }
  pdl_wait_then_release();

  if (warp == 0) {
    if (elect_one()) {
      uint32_t stage = 0, phase = 0;
      const uint64_t pol_x = policy_evict_last();
      for (int kb = k0; kb < k1; ++kb) {
        if (!wait_phase(&empty[stage], phase ^ 1u, abort_flag, p.status)) break;
        const uint32_t sf = (uint32_t)min(2, p.chunks - 2 * kb) * kMxTile;
        if (kb - k0 >= early) load_w(kb, stage);
        if (!QUANT) {
          tma_load_2d(sm_b + stage * S::kB, &tm_x, &full[stage], kb * (int)kRowBytes, tok0, pol_x);
          bulk_load(sm_sf + (stage * 2 + 1) * kSfBytes,
                    p.x_scales + ((size_t)(tok0 >> 7) * p.chunks + 2 * kb) * kMxTile, sf,
                    &full[stage]);
        }
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
      }
      // the loads in flight land before the block leaves
      for (int s = 0; s < STAGES; ++s) {
        const uint32_t issued = s < (int)stage ? phase : phase ^ 1u;
        drain_bar(&full[s], issued, p.status);
      }
    }
  } else if (warp == 1) {
    if (elect_one()) {
      uint32_t stage = 0, phase = 0;
      bool ok = !QUANT || wait_phase(x_full, 0, abort_flag, p.status);
      for (int kb = k0; ok && kb < k1; ++kb) {
        if (!wait_phase(&full[stage], phase, abort_flag, p.status)) { ok = false; break; }
        tc_fence_after();
        const int n64 = min(4, (p.K - kb * kStageK + 63) >> 6);  // of K there is
        const uint32_t sf = tmem + S::kSfCol + (uint32_t)(kb & 1) * 16;
        const uint32_t sa = smem_u32(sm_sf + stage * (QUANT ? 1 : 2) * kSfBytes);
        const uint32_t xb = QUANT ? smem_u32(sm_x + (kb - k0) * S::kB)
                                  : smem_u32(sm_b + stage * S::kB);
        const uint32_t sb = QUANT ? smem_u32(sm_x + nx * S::kB + (kb - k0) * kSfBytes)
                                  : sa + kSfBytes;
        for (int c = 0; 2 * c < n64; ++c) {
          tmem_cp_scales(sf + 4 * c, scale_desc(sa + c * kMxTile));
          tmem_cp_scales(sf + 8 + 4 * c, scale_desc(sb + c * kMxTile));
        }
        const uint64_t ad = sw128_desc(smem_u32(smem + stage * S::kA));
        const uint64_t bd = sw128_desc(xb);
        for (int j = 0; j < n64; ++j)
          mma_mxf4(tmem, ad + 2 * j, bd + 2 * j, idesc_mxf4(kBM, npad, 2 * (j & 1)),
                   sf + 4 * (j >> 1), sf + 8 + 4 * (j >> 1), (kb > k0 || j) ? 1u : 0u);
        mma_commit(&empty[stage]);
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
      }
      if (ok) mma_commit(acc_full);
      // where a wait gave up, the MMAs that were issued end before the block leaves
      for (int s = 0; !ok && s < STAGES; ++s)
        drain_bar(&empty[s], s < (int)stage ? phase : phase ^ 1u, p.status);
    }
  } else {
    const int w = warp - 2;
    if (QUANT) {
      // Rows of 256 of K, one a warp at a time, all of the block's loads on their way at once (behind the
      // weights' loads a second batch would wait for microseconds), into swizzled tiles and their scales;
      // one fence and one arrival for the whole of x.
      const int rows = ntok * (k1 - k0);  // row q: token q % ntok of stage q / ntok
      const uint32_t inv = 65536u / (uint32_t)ntok + 1;  // q < 64, exact
      uint4 u[kQuantRows];
#pragma unroll
      for (int i = 0; i < kQuantRows; ++i) {
        const int q = w + 4 * i, kb = (int)(((uint32_t)q * inv) >> 16), n = q - kb * ntok;
        const int k = (k0 + kb) * kStageK + 8 * lane;
        u[i] = make_uint4(0, 0, 0, 0);
        if (q < rows && k < p.K) u[i] = ldg_u4(p.x + (int64_t)(tok0 + n) * p.x_stride + k);
      }
#pragma unroll
      for (int i = 0; i < kQuantRows; ++i) {
        const int q = w + 4 * i, kb = (int)(((uint32_t)q * inv) >> 16), n = q - kb * ntok;
        if (q >= rows) break;
        float v[8];
        mxq::bf16x8(u[i], v);
        uint32_t s;
        const uint32_t c = mxq::quantise8(v, s);
        *reinterpret_cast<uint32_t*>(sm_x + kb * S::kB + n * kRowBytes +
                                     (((lane >> 2) ^ (n & 7)) << 4) + (lane & 3) * 4) = c;
        if ((lane & 3) == 0) {
          const int j = lane >> 2;
          sm_x[nx * S::kB + kb * kSfBytes + (j >> 2) * kMxTile + (n & 31) * 16 + (n >> 5) * 4 +
               (j & 3)] = (uint8_t)s;
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(x_full);
    }
    // the sums: lane = row of w, column = token
    if (__all_sync(0xffffffffu, wait_phase(acc_full, 0, abort_flag, p.status))) {
      tc_fence_after();
      const int qd = warp & 3;
      float* part = reinterpret_cast<float*>(smem) + qd * 32 + lane;
      for (int c0 = 0; c0 < npad; c0 += 16) {
        uint32_t r[16];
        tmem_ld16(tmem + ((uint32_t)(qd * 32) << 16) + c0, r);
        tmem_ld_wait(r);
#pragma unroll
        for (int j = 0; j < 16; ++j) part[(c0 + j) * kBM] = __uint_as_float(r[j]);
      }
      tc_fence_before();
    }
  }
  __syncwarp();
  if (p.splits > 1) cluster_sync();
  else __syncthreads();

  // rank r of the cluster finishes its share of the tile's sums, four rows of w at a time
  {
    const int total = ntok * (kBM / 4);
    const int q1 = (int)((long)total * (rank + 1) / p.splits);
    const uint32_t base = smem_u32(smem);
    for (int q = (int)((long)total * rank / p.splits) + threadIdx.x; q < q1; q += kLinThreads) {
      const int n = q >> 5, feat = row0 + 4 * (q & 31);
      if (feat >= p.N) continue;
      const float4 a = p.splits == 1   ? *reinterpret_cast<const float4*>(smem + 16 * q)
                       : p.splits == 2 ? gathered<2>(base + 16 * q)
                       : p.splits == 4 ? gathered<4>(base + 16 * q)
                                       : gathered<8>(base + 16 * q);
      float v[4] = {a.x, a.y, a.z, a.w};
      uint16_t* y = p.y + (int64_t)(tok0 + n) * p.y_stride + feat;
      const uint16_t* res = p.residual + (int64_t)(tok0 + n) * p.r_stride + feat;
      if (p.bias) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += feat + i < p.N ? __ldg(p.bias + feat + i) : 0.f;
      }
      if (p.vec && feat + 3 < p.N) {
        if (p.residual) {
          const uint2 r = *reinterpret_cast<const uint2*>(res);
          v[0] = with_residual(v[0], (uint16_t)r.x);
          v[1] = with_residual(v[1], (uint16_t)(r.x >> 16));
          v[2] = with_residual(v[2], (uint16_t)r.y);
          v[3] = with_residual(v[3], (uint16_t)(r.y >> 16));
        }
        uint2 o;
        o.x = f32_to_bf16_rn(v[0]) | (uint32_t)f32_to_bf16_rn(v[1]) << 16;
        o.y = f32_to_bf16_rn(v[2]) | (uint32_t)f32_to_bf16_rn(v[3]) << 16;
        *reinterpret_cast<uint2*>(y) = o;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (feat + i < p.N)
            y[i] = f32_to_bf16_rn(p.residual ? with_residual(v[i], res[i]) : v[i]);
      }
    }
  }
  __syncwarp();
  if (p.splits > 1) cluster_sync();  // no block leaves while another reads its sums
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, S::kCols);
  }
}

template <int NT, int STAGES, bool QUANT>
cudaError_t launch_tile(const CUtensorMap& w, const CUtensorMap& x, const LinParams& p, int tiles,
                        cudaStream_t st) {
  using S = LinSmem<NT, STAGES, QUANT>;
  const int nst = (p.chunks + 1) / 2;
  const uint32_t smem = S::total(QUANT ? (nst + p.splits - 1) / p.splits : 0);
  auto kern = k_mx_linear<NT, STAGES, QUANT>;
  // the most that any call takes: calls of several host threads do not lower it for each other
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)S::total(QUANT ? kQuantStages : 0));
  if (e != cudaSuccess) return e;
  count_launches(1);
  const dim3 grid((unsigned)tiles * (unsigned)p.splits), block(kLinThreads);
  return p.splits > 1
             ? launch_pdl_cluster(kern, grid, block, smem, st, (unsigned)p.splits, w, x, p)
             : launch_pdl(kern, grid, block, smem, st, w, x, p);
}

// Whether CTA pairs take the product: for more than 128 tokens, but where few tiles have long rows, which pairs
// cannot split. Microseconds fitted to x in MXFP4: pairs 3.1 + 0.265 a stage and wave; split tiles 5.3 to 8.5 by the
// share of the SMs that they fill, and 0.45 a stage of a block. (160 tokens of 128 x 16384: 7.7 by split tiles,
// 20.0 by pairs; of 4096 x 16384: 14.7 and 21.0; of 4096 x 4096: 9.1 and 7.7.)
bool by_pairs(const MxDims& d, int tiles, int splits) {
  if (d.T <= 128) return false;
  const int nst = (mx_chunks(d.K) + 1) / 2, blocks = tiles * splits, sms = num_sms();
  const long pair_tiles = (long)((d.T + 255) / 256) * ((d.N + 127) / 128);
  const long waves = (pair_tiles + sms / 2 - 1) / (sms / 2);
  const float pairs = 3.1f + 0.265f * (float)nst * (float)waves;
  const float split = (2 * blocks <= sms ? 5.3f : blocks <= sms ? 6.5f : 8.5f) +
                      0.45f * (float)((nst + splits - 1) / splits);
  return blocks > 2 * sms || split + 0.5f >= pairs;
}

}  // namespace

cudaError_t launch_mx_linear(const MxDims& d, const void* x, const uint8_t* x_scales,
                             const uint8_t* w, const uint8_t* w_scales, const float* bias,
                             const uint16_t* residual, uint16_t* y, char* ws, const MxWs& L,
                             cudaStream_t st) {
  if (d.T == 0) return cudaSuccess;
  cudaError_t e = cudaSuccess;
  const int nt = d.T <= 16 ? 16 : d.T <= 32 ? 32 : d.T <= 64 ? 64 : 128;
  const int mtiles = (d.N + kBM - 1) / kBM, tiles = mtiles * ((d.T + nt - 1) / nt);
  const int nst = (mx_chunks(d.K) + 1) / 2;
  // Splits along K while all blocks stay resident together, two an SM (of clusters of 4 and 8 the GPU holds
  // 74 and 36 then). Measured at one token of 9216 x 7168: 4 splits 7.5 us, 2 splits 9.2; a second wave of
  // blocks doubles the time. Wide tiles gather more sums and want two stages a block (128 tokens, 2048 x 2048: 8
  // splits of one stage 7.9 us, 4 splits 6.1).
  const int least = nt >= 64 ? 2 : 1;
  int splits = 1;
  while (splits < 8 && 2 * splits * least <= nst &&
         tiles * 2 * splits <= 2 * num_sms() - (splits == 4 ? 16 : splits == 2 ? 8 : 0))
    splits *= 2;
  // The product's own warps quantise x where it is that small, so that a call is one launch: one token of
  // 7168 x 7168 7.0 us against 8.1 with a launch ahead; 8 tokens 9.7 against 8.1, as every block quantises its
  // part of x for itself.
  const int nx = (nst + splits - 1) / splits;
  const bool fused = !d.quantised && nt == 16 && nx <= kQuantStages && d.T * nx <= 4 * kQuantRows;
  const uint8_t* codes = static_cast<const uint8_t*>(x);
  if (!d.quantised && !fused) {
    const MxRows r{d.T, d.K, false, true, d.x_stride};
    uint8_t* c = reinterpret_cast<uint8_t*>(ws + L.codes);
    uint8_t* s = reinterpret_cast<uint8_t*>(ws + L.scales);
    if ((e = launch_mx_quantize(r, x, c, s, st)) != cudaSuccess) return e;
    codes = c;
    x_scales = s;
  }
  LinParams p{};
  p.T = d.T;
  p.N = d.N;
  p.K = d.K;
  p.mtiles = mtiles;
  p.splits = splits;
  p.chunks = mx_chunks(d.K);
  p.x_stride = d.x_stride;
  p.y_stride = d.y_stride;
  p.r_stride = d.r_stride;
  p.x = fused ? static_cast<const uint16_t*>(x) : nullptr;
  p.x_scales = x_scales;
  p.w_scales = w_scales;
  p.bias = bias;
  p.residual = residual;
  p.y = y;
  p.vec = d.y_stride % 4 == 0 && (!residual || d.r_stride % 4 == 0);
  p.early = !d.quantised && !fused;
  p.status = reinterpret_cast<int*>(ws + L.status);
  if (by_pairs(d, tiles, splits)) {
    p.vec = d.y_stride % 8 == 0 && (!residual || d.r_stride % 8 == 0);
    return launch_pair(p, codes, w, st);
  }
  CUtensorMap mw, mx;
  if ((e = encode_u8_2d(&mw, w, d.N, d.K / 2, kBM)) != cudaSuccess) return e;
  mx = mw;
  if (!fused && (e = encode_u8_2d(&mx, codes, d.T, d.K / 2, nt)) != cudaSuccess) return e;
  if (nt == 16)
    return fused ? launch_tile<16, 4, true>(mw, mx, p, tiles, st)
                 : launch_tile<16, 4, false>(mw, mx, p, tiles, st);
  if (nt == 32) return launch_tile<32, 4, false>(mw, mx, p, tiles, st);
  if (nt == 64) return launch_tile<64, 4, false>(mw, mx, p, tiles, st);
  return launch_tile<128, 3, false>(mw, mx, p, tiles, st);
}

}  // namespace moe
