// The MXFP4 product for many tokens: a persistent GEMM on CTA pairs (tcgen05.mma.cta_group::2).
//
// A tile is 256 tokens x BN features, K in stages of 256. The tokens are the M side, so that a thread of
// the epilogue holds a run of consecutive features of one token. Each CTA of the pair loads its own 128
// tokens and half of the tile's weight rows; the scales of all BN weight rows go to both.
//
//   warp 0     TMA: codes and scales of both sides, all completing on the even CTA's stage barrier
//   warp 1     (even CTA) scales to TMEM (tcgen05.cp), four MMAs of 64 of K a stage
//   warps 2-9  epilogue: a lane quadrant and half of the features each. The sums leave TMEM for registers at
//              once and TMEM is handed back before anything is done with them: with one accumulator of 256
//              columns beside the scales' the next tile's MMAs wait for that alone. Then bias and residual,
//              one rounding, boxes of 32 tokens x 64 features stored by TMA (rows that no tensor map takes:
//              store_rows). Stored from registers, 16 bytes a lane, the boxes took the L2 from the loads:
//              a tile's MMAs waited 6000 cycles for operands, 1700 since.
//
// What bounds it: the MMAs. 16384 tokens of 9216 x 7168 (x in MXFP4): 293 us, 7.4 PFLOP/s, the tensor pipe active 82%
// of the time, at the card's power limit; a stage of 256 of K takes 496 cycles where its operands are there
// (124 an MMA of 256 x 256 x 64), a tile's end 1000 cycles from the last MMA to the next tile's first.
#include "mx_linear.cuh"

namespace moe {
namespace mxl {
namespace {

constexpr int kPairThreads = 320;
constexpr uint32_t kOutBytes = 32 * 128;  // 32 tokens x 64 features of bf16, one swizzle row a token

template <int BN, int STAGES>
struct PairSmem {
  static constexpr uint32_t kA = kBM * kRowBytes;          // this CTA's tokens
  static constexpr uint32_t kB = BN / 2 * kRowBytes;       // its half of the weight rows
  static constexpr uint32_t kTileBytes = kA + kB;
  static constexpr int kBlocks = BN / 128;                 // 128-row blocks of weight scales
  static constexpr uint32_t kSf = (1 + kBlocks) * kSfBytes;
  static constexpr uint32_t kStageBytes = kTileBytes + kSf;
  static constexpr uint32_t kOut = 8 * kOutBytes;          // a box of the output for each epilogue warp
  static constexpr uint32_t kBias = 8 * BN / 2 * 4;        // and the bias of its features
  static constexpr uint32_t kBars = 8 * (2 * STAGES + 2 + 8) + 16;
  static constexpr uint32_t kTotal = STAGES * kStageBytes + kOut + kBias + kBars + 1024;
  static constexpr uint32_t kSfCols = 8 + 8 * kBlocks;     // of a stage: tokens, then weights
};

// Two values rounded to bf16, the first in the low half.
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Element e of token r in a box.
__device__ __forceinline__ uint16_t* boxed(uint8_t* box, int r, int e) {
  return reinterpret_cast<uint16_t*>(box + r * 128 + (((e >> 3) ^ (r & 7)) << 4) + (e & 7) * 2);
}

// A box of 32 tokens x 64 features to rows that no tensor map takes, a token at a time: words where they
// are aligned; in a row that starts at an odd element the words are of a lane's second element and the next
// lane's first, and the row's ends go out as single elements. Few instructions a row, and predicates instead of
// branches: eight warps an SM wait for each of them.
template <bool ALL>
__device__ __forceinline__ void store_rows(const LinParams& p, uint8_t* box, int tok0, int f0,
                                           int lane) {
  const int rows = ALL ? 32 : min(32, p.T - tok0);
  const int64_t step = p.y_stride * 2;
  uint8_t* o = reinterpret_cast<uint8_t*>(p.y + (int64_t)tok0 * p.y_stride + f0 + 2 * lane);
  const uint32_t flip = (uint32_t)p.y_stride & 1u;
  uint32_t odd = (uint32_t)(reinterpret_cast<uintptr_t>(o) >> 1) & 1u;
  const bool end = lane == 0 || lane == 31;
  const uint32_t shift = lane ? 16 : 0, at = lane ? 2 : 0;  // of the single element that an end's lane has
#pragma unroll
  for (int r0 = 0; r0 < 32; r0 += 8) {
    uint32_t a[8], next[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = *reinterpret_cast<const uint32_t*>(boxed(box, r0 + i, 2 * lane));
#pragma unroll
    for (int i = 0; i < 8; ++i) next[i] = __shfl_down_sync(0xffffffffu, a[i], 1);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool there = ALL || r0 + i < rows;
      const uint32_t w = __byte_perm(a[i], next[i], odd ? 0x5432 : 0x3210);
      if (there && (lane < 31 || !odd)) *reinterpret_cast<uint32_t*>(o + 2 * odd) = w;
      if (there && odd && end) *reinterpret_cast<uint16_t*>(o + at) = (uint16_t)(a[i] >> shift);
      odd ^= flip;
      o += step;
    }
  }
}

// The residual of such rows into a box, 16 loads of 32 elements at a time (aligned words and single ends, half as
// many loads, took longer: eight rows at a time instead of these).
__device__ __forceinline__ void load_rows(const LinParams& p, uint8_t* box, int tok0, int f0,
                                          int lane) {
  for (int r0 = 0; r0 < 32; r0 += 8) {
    uint16_t a[8][2];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int r = r0 + (i >> 1), e = lane + 32 * (i & 1);
      a[i >> 1][i & 1] = tok0 + r < p.T && f0 + e < p.N
                             ? p.residual[(int64_t)(tok0 + r) * p.r_stride + f0 + e]
                             : (uint16_t)0;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) *boxed(box, r0 + (i >> 1), lane + 32 * (i & 1)) = a[i >> 1][i & 1];
  }
}

// store_rows where fewer than 64 features are left.
__device__ __forceinline__ void store_columns(const LinParams& p, uint8_t* box, int tok0, int f0,
                                              int lane) {
  const int rows = min(32, p.T - tok0), cols = p.N - f0;
  uint16_t* o = p.y + (int64_t)tok0 * p.y_stride + f0 + 2 * lane;
  for (int r = 0; r < rows; ++r, o += p.y_stride) {
    const uint32_t a = *reinterpret_cast<const uint32_t*>(boxed(box, r, 2 * lane));
    if (2 * lane < cols) o[0] = (uint16_t)a;
    if (2 * lane + 1 < cols) o[1] = (uint16_t)(a >> 16);
  }
}

template <int BN, int STAGES, bool RES>
__global__ void __launch_bounds__(kPairThreads, 1)
    k_mx_linear_pair(const __grid_constant__ CUtensorMap tm_x,
                     const __grid_constant__ CUtensorMap tm_w,
                     const __grid_constant__ CUtensorMap tm_xs,
                     const __grid_constant__ CUtensorMap tm_ws,
                     const __grid_constant__ CUtensorMap tm_y,
                     const __grid_constant__ CUtensorMap tm_r, const LinParams p, int ttiles,
                     int ftiles) {
  using S = PairSmem<BN, STAGES>;
  static_assert(BN == 128 || BN == 256, "MMA N");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* sm_out = smem + STAGES * S::kTileBytes;
  uint8_t* sm_sf = sm_out + S::kOut;
  float* sm_bias = reinterpret_cast<float*>(sm_sf + STAGES * S::kSf);
  uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(sm_bias) + S::kBias);
  uint64_t* empty = full + STAGES;
  uint64_t* acc_full = empty + STAGES;
  uint64_t* acc_empty = acc_full + 1;
  uint64_t* res_full = acc_empty + 1;  // of each epilogue warp: its residual has landed
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(res_full + 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank();
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);   // the even CTA's loading thread, and both CTAs' bytes
      mbar_init(&empty[s], 1);  // the commit of the stage's MMAs
    }
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, 16);  // the epilogue warps of both CTAs
    for (int w = 0; w < 8; ++w) mbar_init(&res_full[w], 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tm_x);
    prefetch_tmap(&tm_w);
    prefetch_tmap(&tm_xs);
    prefetch_tmap(&tm_ws);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_holder, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers are initialised before either signals the other
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const int tile0 = (int)(blockIdx.x >> 1), tstep = (int)(gridDim.x >> 1);
  const int total = ttiles * ftiles;
  const int nst = (p.chunks + 1) >> 1;

  // A stage's weights and their scales; the even CTA's thread also announces all of both CTAs' bytes.
  const auto load_w = [&](int tile, int kb, uint32_t stage) {
    const int ft = tile % ftiles, ws = ft * S::kBlocks * p.chunks;
    const uint32_t bar = mapa_shared(smem_u32(&full[stage]), 0);
    const uint64_t pol = policy_evict_normal();
    uint8_t* sf = sm_sf + stage * S::kSf + kSfBytes;
    if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * S::kStageBytes);
    tma_load_2d_pair(smem + stage * S::kTileBytes + S::kA, &tm_w, bar, kb * (int)kRowBytes,
                     ft * BN + rank * (BN / 2), pol);
    // boxes of two 512-byte blocks; beyond K or the last row they hold anything, or zeros
#pragma unroll
    for (int b = 0; b < S::kBlocks; ++b)
      tma_load_2d_pair(sf + b * kSfBytes, &tm_ws, bar, 0, ws + b * p.chunks + 2 * kb, pol);
  };
  // Behind the call's own quantisation of x, which has waited for everything before it, the first
  // stages' weights need not wait for x.
  const int early = p.early && tile0 < total ? min(STAGES, nst) : 0;
  // (Without it, the first stages' way to L2 alone: what the kernel ahead still writes is written there.)
  if (warp == 0 && elect_one() && tile0 < total) {
    for (int kb = 0; kb < early; ++kb) load_w(tile0, kb, (uint32_t)kb);
    const int feat = tile0 % ftiles * BN + rank * (BN / 2);
    for (int kb = early; kb < min(STAGES, nst); ++kb)
      tma_prefetch_2d(&tm_w, kb * (int)kRowBytes, feat);
  }
  pdl_wait_then_release();

  if (warp == 0) {
    if (elect_one()) {
      const uint64_t pol = policy_evict_normal();
      const uint32_t full0 = mapa_shared(smem_u32(&full[0]), 0);
      uint32_t stage = 0, phase = 0;
      bool ok = true;
      for (int tile = tile0; ok && tile < total; tile += tstep) {
        const int tt = tile / ftiles;
        const int tok = tt * 256 + rank * 128, xs = (tt * 2 + rank) * p.chunks;
        for (int kb = 0; kb < nst; ++kb) {
          if (!wait_phase(&empty[stage], phase ^ 1u, abort_flag, p.status)) { ok = false; break; }
          if (tile != tile0 || kb >= early) load_w(tile, kb, stage);
          const uint32_t bar = full0 + 8u * stage;
          tma_load_2d_pair(smem + stage * S::kTileBytes, &tm_x, bar, kb * (int)kRowBytes, tok, pol);
          tma_load_2d_pair(sm_sf + stage * S::kSf, &tm_xs, bar, 0, xs + 2 * kb, pol);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      // the loads in flight land, and the commits for both CTAs' stages arrive, before a CTA leaves
      for (int s = 0; s < STAGES; ++s) {
        const uint32_t issued = s < (int)stage ? phase : phase ^ 1u;
        if (rank == 0) drain_bar(&full[s], issued, p.status);
        drain_bar(&empty[s], issued, p.status);
      }
    }
  } else if (warp == 1) {
    // one elected thread: under a comparison of lane numbers a stage's MMAs took 1.5 times as long
    if (rank == 0 && elect_one()) {
      uint32_t stage = 0, phase = 0, it = 0, acc_phase = 0;
      bool ok = true;
      for (int tile = tile0; ok && tile < total; tile += tstep) {
        if (!wait_phase(acc_empty, acc_phase ^ 1u, abort_flag, p.status)) break;
        tc_fence_after();
        for (int kb = 0; kb < nst; ++kb, ++it) {
          if (!wait_phase(&full[stage], phase, abort_flag, p.status)) { ok = false; break; }
          tc_fence_after();
          const int n64 = min(4, (p.K - kb * kStageK + 63) >> 6);
          const uint32_t sfa = tmem + BN + (it & 1) * S::kSfCols, sfb = sfa + 8;
          const uint32_t sm = smem_u32(sm_sf + stage * S::kSf);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            if (2 * c >= n64) break;
            tmem_cp_scales_pair(sfa + 4 * c, scale_desc(sm + c * kMxTile));
#pragma unroll
            for (int b = 0; b < S::kBlocks; ++b)
              tmem_cp_scales_pair(sfb + c * 4 * S::kBlocks + 4 * b,
                                  scale_desc(sm + (1 + b) * kSfBytes + c * kMxTile));
          }
          const uint32_t st = smem_u32(smem + stage * S::kTileBytes);
          const uint64_t ad = sw128_desc(st), bd = sw128_desc(st + S::kA);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (j >= n64) break;
            mma_mxf4_pair(tmem, ad + 2 * j, bd + 2 * j, idesc_mxf4(256, BN, 2 * (j & 1)),
                          sfa + 4 * (j >> 1), sfb + (j >> 1) * 4 * S::kBlocks,
                          (kb | j) ? 1u : 0u);
          }
          mma_commit_pair(&empty[stage]);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        mma_commit_pair(acc_full);
        acc_phase ^= 1u;
      }
    }
  } else {
    const int qd = warp & 3, half = (warp - 2) >> 2;
    constexpr int kCols = BN / 2;  // features of a thread
    const uint32_t empty0 = mapa_shared(smem_u32(acc_empty), 0);
    uint8_t* box = sm_out + (warp - 2) * kOutBytes;
    uint8_t* my = box + lane * 128;
    float* bias = sm_bias + (warp - 2) * kCols;
    uint64_t* rbar = &res_full[warp - 2];
    uint32_t acc_phase = 0, res_phase = 0;
    for (int tile = tile0; tile < total; tile += tstep) {
      const int tt = tile / ftiles, ft = tile - tt * ftiles;
      const int tok0 = tt * 256 + rank * 128 + qd * 32;
      const int feat = ft * BN + half * kCols;
      // the residual of 64 features into the box, once the store before it has been read
      const auto fetch = [&](int f0) {
        if (!RES || tok0 >= p.T || f0 >= p.N) return;
        if (p.vec) {
          if (lane == 0) {
            bulk_wait_read();
            mbar_arrive_expect_tx(rbar, kOutBytes);
            tma_load_2d(box, &tm_r, rbar, f0, tok0, policy_evict_first());
          }
        } else {
          __syncwarp();
          load_rows(p, box, tok0, f0, lane);
          __syncwarp();
        }
      };
      fetch(feat);
      if (p.bias) {  // to shared memory while the sums are formed
        __syncwarp();
        for (int i = lane; i < kCols; i += 32) bias[i] = feat + i < p.N ? __ldg(p.bias + feat + i) : 0.f;
        __syncwarp();
      }
      bool ok = __all_sync(0xffffffffu, wait_phase(acc_full, acc_phase, abort_flag, p.status));
      if (!ok) {
        if (RES && p.vec && tok0 < p.T && feat < p.N) drain_bar(rbar, res_phase, p.status);
        break;
      }
      acc_phase ^= 1u;
      tc_fence_after();
      uint32_t r[kCols];
#pragma unroll
      for (int c = 0; c < kCols; c += 32)
        tmem_ld32(tmem + ((uint32_t)(qd * 32) << 16) + half * kCols + c, r + c);
#pragma unroll
      for (int c = 0; c < kCols; c += 32) tmem_ld_wait32(r + c);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(empty0);
#pragma unroll
      for (int h = 0; h < kCols / 64; ++h) {
        const int f0 = feat + 64 * h;
        if (tok0 >= p.T || f0 >= p.N) break;
        if (h) fetch(f0);
        if (RES && p.vec) {
          ok = __all_sync(0xffffffffu, wait_phase(rbar, res_phase, abort_flag, p.status));
          if (!ok) {  // the box in flight lands before the CTA leaves; nothing of it is stored
            drain_bar(rbar, res_phase, p.status);
            break;
          }
          res_phase ^= 1u;
        } else if (p.vec) {
          if (lane == 0) bulk_wait_read();
          __syncwarp();
        } else {
          __syncwarp();
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) {  // 8 features
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[64 * h + 8 * c + i]);
          if (p.bias) {
            const float4 a = *reinterpret_cast<const float4*>(bias + 64 * h + 8 * c);
            const float4 b = *reinterpret_cast<const float4*>(bias + 64 * h + 8 * c + 4);
            v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
            v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
          }
          uint4* at = reinterpret_cast<uint4*>(my + ((c ^ (lane & 7)) << 4));
          if (RES) {
            const uint4 u = *at;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += bf16x8_elem(u, i);
          }
          *at = make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]),
                           bf16_pair(v[6], v[7]));
        }
        if (p.vec) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) tma_store_2d(&tm_y, box, f0, tok0);  // rows and columns beyond y are cut
        } else {
          __syncwarp();
          if (f0 + 64 > p.N) store_columns(p, box, tok0, f0, lane);
          else if (tok0 + 32 <= p.T) store_rows<true>(p, box, tok0, f0, lane);
          else store_rows<false>(p, box, tok0, f0, lane);
          __syncwarp();
        }
      }
      if (!ok) break;
    }
    if (p.vec && lane == 0) bulk_wait_all();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no CTA leaves while its peer may still signal it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// Scales in tiles as rows of 512 bytes, boxes of two rows, as they lie.
cudaError_t encode_scales(CUtensorMap* m, const uint8_t* base, uint64_t blocks) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {kMxTile / 4, blocks};
  const cuuint64_t strides[1] = {kMxTile};
  const cuuint32_t box[2] = {kMxTile / 4, 2};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<uint8_t*>(base), dims,
                        strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// [rows, cols] bf16 whose rows lie `stride` elements apart, boxes of 32 rows x 64 columns.
cudaError_t encode_out(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols,
                       int64_t stride) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {(cuuint64_t)stride * 2};
  const cuuint32_t box[2] = {64, 32};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims,
                        strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int BN, int STAGES, bool RES>
cudaError_t launch_bn(const LinParams& p, const uint8_t* codes, const uint8_t* w,
                      cudaStream_t st) {
  using S = PairSmem<BN, STAGES>;
  static_assert(S::kTotal <= 227 * 1024, "shared memory");
  static_assert(BN + 2 * S::kSfCols <= 512, "TMEM columns");
  CUtensorMap mx, mw, mxs, mws;
  cudaError_t e = encode_u8_2d(&mx, codes, p.T, p.K / 2, 128);
  if (e == cudaSuccess) e = encode_u8_2d(&mw, w, p.N, p.K / 2, BN / 2);
  if (e == cudaSuccess) e = encode_scales(&mxs, p.x_scales, (uint64_t)((p.T + 127) / 128) * p.chunks);
  if (e == cudaSuccess) e = encode_scales(&mws, p.w_scales, (uint64_t)((p.N + 127) / 128) * p.chunks);
  if (e != cudaSuccess) return e;
  CUtensorMap my = mx, mr = mx;  // not used where the rows do not suit a tensor map
  if (p.vec) {
    e = encode_out(&my, p.y, p.T, p.N, p.y_stride);
    if (e == cudaSuccess && RES) e = encode_out(&mr, p.residual, p.T, p.N, p.r_stride);
    if (e != cudaSuccess) return e;
  }
  auto kern = k_mx_linear_pair<BN, STAGES, RES>;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kTotal);
  if (e != cudaSuccess) return e;
  const int ttiles = (p.T + 255) / 256, ftiles = (p.N + BN - 1) / BN;
  const long total = (long)ttiles * ftiles;
  const long pairs = num_sms() / 2;
  count_launches(1);
  return launch_pdl_cluster(kern, dim3((unsigned)(2 * (total < pairs ? total : pairs))),
                            dim3(kPairThreads), S::kTotal, st, 2u, mx, mw, mxs, mws, my, mr, p,
                            ttiles, ftiles);
}

}  // namespace

cudaError_t launch_pair(const LinParams& p, const uint8_t* codes, const uint8_t* w,
                        cudaStream_t st) {
  // 256 features a tile, or 128 where that makes the longest pair's share of tiles shorter. A tile's
  // time in stages of 256 features' (496 cycles): 0.87 a stage with 128 (the tokens' side bounds the MMAs),
  // and its ends
  const long pairs = num_sms() / 2, tt = (p.T + 255) / 256;
  const float nst = (float)((p.chunks + 1) / 2);
  const float t256 = (float)((tt * ((p.N + 255) / 256) + pairs - 1) / pairs) * (nst + 5.f);
  const float t128 = (float)((tt * ((p.N + 127) / 128) + pairs - 1) / pairs) * (0.87f * nst + 3.f);
  if (t128 < t256)
    return p.residual ? launch_bn<128, 7, true>(p, codes, w, st)
                      : launch_bn<128, 7, false>(p, codes, w, st);
  return p.residual ? launch_bn<256, 5, true>(p, codes, w, st)
                    : launch_bn<256, 5, false>(p, codes, w, st);
}

}  // namespace mxl
}  // namespace moe
