// Quantisation of matrices to MXFP4, the values back, and scales from rows to tiles.
//
// Each element is read once and written once: the kernels are bound by HBM for all but small matrices (32768 x
// 7168 bf16: 92 us there, 0.95 of the copy rate, 88 us back, 0.99), and by launch latency for those (256 x 7168:
// 1.8 and 2.1 us). A thread takes 16 consecutive elements to quantise (two lanes a block of 32: one exchange for
// its largest magnitude), 8 to read back (32 lanes store 512 bytes of bf16 in a row).
#include "mx_quant.cuh"

namespace moe {
namespace {

using namespace mxq;

// Sixteen elements.
template <bool F32>
__device__ __forceinline__ void load16(const void* x, int64_t at, float (&v)[16]) {
  if (F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 a = ld_stream_u4(static_cast<const float*>(x) + at + 4 * i);
      v[4 * i] = __uint_as_float(a.x);
      v[4 * i + 1] = __uint_as_float(a.y);
      v[4 * i + 2] = __uint_as_float(a.z);
      v[4 * i + 3] = __uint_as_float(a.w);
    }
  } else {
    const uint4 a = ld_stream_u4(static_cast<const uint16_t*>(x) + at);
    const uint4 b = ld_stream_u4(static_cast<const uint16_t*>(x) + at + 8);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = bf16x8_elem(a, i);
      v[8 + i] = bf16x8_elem(b, i);
    }
  }
}

// A block takes consecutive units of its slab of kSlab rows (blockIdx.y). Places are 32-bit within a slab, divided
// by multiplication: a 64-bit division a unit took twice the time of the rest.
constexpr int kQuantThreads = 256;  // of a block (32768 x 7168: 92 us, 128 threads 116, 512 threads 94)
constexpr int kBackThreads = 128;   // (88 us, 256 threads 93, 512 threads 97)
constexpr int kSlab = 1 << 16;

struct MxWalk {
  long rows;
  int K, chunks;
  int64_t stride;
  FastDiv per;  // units of a row
};

__device__ __forceinline__ uint32_t divided(uint32_t n, const FastDiv& f) {
  return (uint32_t)(((uint64_t)n * f.m) >> f.p);
}

// Units of 16 elements: half a block of 32. WORDS (K a multiple of 128): the scales of four blocks lie in 8
// lanes and go out as a word.
template <bool F32, bool TILES, bool WORDS>
__global__ void __launch_bounds__(kQuantThreads) k_mx_quantize(const void* __restrict__ x,
                                                          const MxWalk a,
                                                          uint8_t* __restrict__ codes,
                                                          uint8_t* __restrict__ scales) {
  pdl_wait_then_release();
  const long r0 = (long)blockIdx.y * kSlab;
  const uint32_t units = (uint32_t)min(a.rows - r0, (long)kSlab) * a.per.d;
  const uint32_t u = blockIdx.x * kQuantThreads + threadIdx.x;
  const int lane = threadIdx.x & 31, blocks = a.K >> 5;
  const uint32_t r = divided(u, a.per), c = u - r * a.per.d;
  const long row = r0 + r;
  float v[16];
  if (u < units) {
    load16<F32>(x, row * a.stride + 16 * c, v);
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = 0.f;
  }
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 16; ++e) m = max(m, __float_as_uint(v[e]) & 0x7FFFFFFFu);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  uint32_t s = scale_byte(m);
  uint2 w = make_uint2(0, 0);
  if (s != 255u) {
    const float f = inverse(s);
    float h[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = v[e] * f;
    w.x = codes8(h);
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = v[8 + e] * f;
    w.y = codes8(h);
  }
  if (WORDS) {
    s |= __shfl_down_sync(0xffffffffu, s, 2) << 8;  // of lanes 0, 8, ..: blocks 0, 1; then 2, 3
    s |= __shfl_down_sync(0xffffffffu, s, 4) << 16;
  }
  if (u >= units) return;
  reinterpret_cast<uint2*>(codes)[row * a.per.d + c] = w;
  const int j = (int)(c >> 1);
  const size_t at = TILES ? tile_at(row, j, a.chunks) : (size_t)row * blocks + j;
  if (WORDS) {
    if ((lane & 7) == 0) *reinterpret_cast<uint32_t*>(scales + at) = s;
  } else if ((lane & 1) == 0) {
    scales[at] = (uint8_t)s;
    if (TILES && j == blocks - 1)  // padding of the last chunk: codes beyond K are taken as 0, times 1
      for (int e = 1; e < 4 - (j & 3); ++e) scales[at + e] = 127;
  }
}

// Units of 8 elements, every kBackThreads-th of the block's to a thread.
template <bool F32, bool TILES, int UNITS>
__global__ void __launch_bounds__(kBackThreads) k_mx_dequantize(const uint8_t* __restrict__ codes,
                                                            const uint8_t* __restrict__ scales,
                                                            const MxWalk a, void* __restrict__ y) {
  pdl_wait_then_release();
  const long r0 = (long)blockIdx.y * kSlab;
  const uint32_t units = (uint32_t)min(a.rows - r0, (long)kSlab) * a.per.d;
  const uint32_t u0 = blockIdx.x * (kBackThreads * UNITS) + threadIdx.x;
  uint32_t w[UNITS], s[UNITS], r[UNITS], c[UNITS];
#pragma unroll
  for (int i = 0; i < UNITS; ++i) {
    const uint32_t u = u0 + kBackThreads * i;
    r[i] = divided(u, a.per);
    c[i] = u - r[i] * a.per.d;
    w[i] = s[i] = 0;
    if (u >= units) continue;
    const long row = r0 + r[i];
    w[i] = __ldg(reinterpret_cast<const uint32_t*>(codes) + row * a.per.d + c[i]);
    s[i] = __ldg(scales + (TILES ? tile_at(row, (int)(c[i] >> 2), a.chunks)
                                 : (size_t)row * (a.K >> 5) + (c[i] >> 2)));
  }
#pragma unroll
  for (int i = 0; i < UNITS; ++i) {
    if (u0 + kBackThreads * i >= units) continue;
    const float f = value(s[i]);
    float v[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 p = pair((w[i] >> (8 * e)) & 0xFFu);
      v[2 * e] = p.x * f;
      v[2 * e + 1] = p.y * f;
    }
    const int64_t at = (r0 + r[i]) * a.stride + 8 * c[i];
    if (F32) {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(y) + at);
      o[0] = make_float4(v[0], v[1], v[2], v[3]);
      o[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      uint4 o;
      o.x = f32_to_bf16_rn(v[0]) | (uint32_t)f32_to_bf16_rn(v[1]) << 16;
      o.y = f32_to_bf16_rn(v[2]) | (uint32_t)f32_to_bf16_rn(v[3]) << 16;
      o.z = f32_to_bf16_rn(v[4]) | (uint32_t)f32_to_bf16_rn(v[5]) << 16;
      o.w = f32_to_bf16_rn(v[6]) | (uint32_t)f32_to_bf16_rn(v[7]) << 16;
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(y) + at) = o;
    }
  }
}

// A thread writes the four scales of a row's chunk.
__global__ void __launch_bounds__(256) k_mx_tile_scales(const uint8_t* __restrict__ scales,
                                                        long rows, int blocks,
                                                        uint8_t* __restrict__ tiles) {
  pdl_wait_then_release();
  const int chunks = (blocks + 3) >> 2;
  const long u = (long)blockIdx.x * blockDim.x + threadIdx.x;
  if (u >= rows * chunks) return;
  const long r = u / chunks;
  const int q = (int)(u - r * chunks);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = 4 * q + i;
    w |= (j < blocks ? (uint32_t)scales[r * blocks + j] : 127u) << (8 * i);
  }
  *reinterpret_cast<uint32_t*>(tiles + tile_at(r, 4 * q, chunks)) = w;
}

}  // namespace

namespace {

MxWalk walk(const MxRows& r, int unit, long block, dim3* grid) {
  MxWalk a{r.rows, r.K, mx_chunks(r.K), r.stride, fast_div((uint32_t)(r.K / unit))};
  const long slab = r.rows < kSlab ? r.rows : kSlab;
  *grid = dim3((unsigned)((slab * (r.K / unit) + block - 1) / block),
               (unsigned)((r.rows + kSlab - 1) / kSlab));
  return a;
}

template <bool F32, bool TILES>
cudaError_t quantize(const MxRows& r, const void* x, uint8_t* codes, uint8_t* scales,
                     cudaStream_t st) {
  dim3 grid;
  const MxWalk a = walk(r, 16, kQuantThreads, &grid);
  return r.K % 128 == 0 ? launch_pdl(k_mx_quantize<F32, TILES, true>, grid, dim3(kQuantThreads), 0, st, x,
                                     a, codes, scales)
                        : launch_pdl(k_mx_quantize<F32, TILES, false>, grid, dim3(kQuantThreads), 0, st, x,
                                     a, codes, scales);
}

template <bool F32, bool TILES>
cudaError_t dequantize(const MxRows& r, const uint8_t* codes, const uint8_t* scales, void* y,
                       cudaStream_t st) {
  dim3 grid;
  // matrices that fill the SMs at a unit a thread get four (32768 x 7168: 95 us with one, 89 with four; in the
  // other direction, where a unit is 32 bytes, one took 94 us, two 105, four 135)
  if (r.rows * (r.K / 8) > (long)num_sms() * 2048) {
    const MxWalk a = walk(r, 8, 4 * kBackThreads, &grid);
    return launch_pdl(k_mx_dequantize<F32, TILES, 4>, grid, dim3(kBackThreads), 0, st, codes, scales, a,
                      y);
  }
  const MxWalk a = walk(r, 8, kBackThreads, &grid);
  return launch_pdl(k_mx_dequantize<F32, TILES, 1>, grid, dim3(kBackThreads), 0, st, codes, scales, a, y);
}

}  // namespace

cudaError_t launch_mx_quantize(const MxRows& r, const void* x, uint8_t* codes, uint8_t* scales,
                               cudaStream_t st) {
  if (r.rows == 0) return cudaSuccess;
  count_launches(1);
  if (r.f32)
    return r.tiles ? quantize<true, true>(r, x, codes, scales, st)
                   : quantize<true, false>(r, x, codes, scales, st);
  return r.tiles ? quantize<false, true>(r, x, codes, scales, st)
                 : quantize<false, false>(r, x, codes, scales, st);
}

cudaError_t launch_mx_dequantize(const MxRows& r, const uint8_t* codes, const uint8_t* scales,
                                 void* y, cudaStream_t st) {
  if (r.rows == 0) return cudaSuccess;
  count_launches(1);
  if (r.f32)
    return r.tiles ? dequantize<true, true>(r, codes, scales, y, st)
                   : dequantize<true, false>(r, codes, scales, y, st);
  return r.tiles ? dequantize<false, true>(r, codes, scales, y, st)
                 : dequantize<false, false>(r, codes, scales, y, st);
}

cudaError_t launch_mx_tile_scales(long rows, int K, const uint8_t* scales, uint8_t* tiles,
                                  cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  const long units = rows * mx_chunks(K);
  count_launches(1);
  return launch_pdl(k_mx_tile_scales, dim3((unsigned)((units + 255) / 256)), dim3(256), 0, st,
                    scales, rows, K / 32, tiles);
}

}  // namespace moe
