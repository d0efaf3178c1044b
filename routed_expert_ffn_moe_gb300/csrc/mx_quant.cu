// Quantisation of matrices to MXFP4, the values back, and scales from rows to tiles.
//
// Each element is read once and written once: the kernels are bound by HBM for all but small matrices,
// and by launch latency for those. A thread takes 8 consecutive elements (16 bytes of bf16), so a warp reads
// 512 bytes in a row and a block of 32 is a quad of lanes, whose largest magnitude takes two exchanges.
#include "mx_quant.cuh"

namespace moe {
namespace {

using namespace mxq;

template <bool F32>
__device__ __forceinline__ void load8(const void* x, int64_t at, float (&v)[8]) {
  if (F32) {
    const uint4 a = ld_stream_u4(static_cast<const float*>(x) + at);
    const uint4 b = ld_stream_u4(static_cast<const float*>(x) + at + 4);
    v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y);
    v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
    v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y);
    v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
  } else {
    bf16x8(ld_stream_u4(static_cast<const uint16_t*>(x) + at), v);
  }
}

// Unit u of 8 elements: row u / (K / 8). The grid covers all units, rounded up to whole warps.
template <bool F32, bool TILES>
__global__ void __launch_bounds__(256) k_mx_quantize(const void* __restrict__ x, long rows, int K,
                                                     int64_t stride, uint8_t* __restrict__ codes,
                                                     uint8_t* __restrict__ scales) {
  pdl_wait_then_release();
  const int per = K >> 3;
  const long u = (long)blockIdx.x * blockDim.x + threadIdx.x;
  const bool there = u < rows * per;
  const long r = there ? u / per : 0;
  const int c = there ? (int)(u - r * per) : 0;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (there) load8<F32>(x, r * stride + 8 * c, v);
  const uint32_t s = quad_scale(v);
  const float f = inverse(s);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = s == 255u ? 0.f : v[i] * f;
  if (!there) return;
  reinterpret_cast<uint32_t*>(codes)[u] = codes8(v);
  if ((c & 3) == 0) {
    const int j = c >> 2, blocks = K >> 5;
    if (!TILES) {
      scales[r * blocks + j] = (uint8_t)s;
    } else {
      const size_t at = tile_at(r, j, mx_chunks(K));
      scales[at] = (uint8_t)s;
      if (j == blocks - 1)  // padding of the last chunk: codes beyond K are taken as 0, times 1
        for (int i = 1; i < 4 - (j & 3); ++i) scales[at + i] = 127;
    }
  }
}

template <bool F32, bool TILES>
__global__ void __launch_bounds__(256) k_mx_dequantize(const uint8_t* __restrict__ codes,
                                                       const uint8_t* __restrict__ scales, long rows,
                                                       int K, int64_t stride, void* __restrict__ y) {
  pdl_wait_then_release();
  const int per = K >> 3;
  const long u = (long)blockIdx.x * blockDim.x + threadIdx.x;
  if (u >= rows * per) return;
  const long r = u / per;
  const int c = (int)(u - r * per), j = c >> 2;
  const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(codes) + u);
  const float f = value(TILES ? scales[tile_at(r, j, mx_chunks(K))] : scales[r * (K >> 5) + j]);
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = pair((w >> (8 * i)) & 0xFFu);
    v[2 * i] = p.x * f;
    v[2 * i + 1] = p.y * f;
  }
  const int64_t at = r * stride + 8 * c;
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

cudaError_t launch_mx_quantize(const MxRows& r, const void* x, uint8_t* codes, uint8_t* scales,
                               cudaStream_t st) {
  if (r.rows == 0) return cudaSuccess;
  const dim3 grid((unsigned)((r.rows * (r.K / 8) + 255) / 256)), block(256);
  count_launches(1);
  if (r.f32)
    return r.tiles ? launch_pdl(k_mx_quantize<true, true>, grid, block, 0, st, x, r.rows, r.K,
                                r.stride, codes, scales)
                   : launch_pdl(k_mx_quantize<true, false>, grid, block, 0, st, x, r.rows, r.K,
                                r.stride, codes, scales);
  return r.tiles ? launch_pdl(k_mx_quantize<false, true>, grid, block, 0, st, x, r.rows, r.K,
                              r.stride, codes, scales)
                 : launch_pdl(k_mx_quantize<false, false>, grid, block, 0, st, x, r.rows, r.K,
                              r.stride, codes, scales);
}

cudaError_t launch_mx_dequantize(const MxRows& r, const uint8_t* codes, const uint8_t* scales,
                                 void* y, cudaStream_t st) {
  if (r.rows == 0) return cudaSuccess;
  const dim3 grid((unsigned)((r.rows * (r.K / 8) + 255) / 256)), block(256);
  count_launches(1);
  if (r.f32)
    return r.tiles ? launch_pdl(k_mx_dequantize<true, true>, grid, block, 0, st, codes, scales,
                                r.rows, r.K, r.stride, y)
                   : launch_pdl(k_mx_dequantize<true, false>, grid, block, 0, st, codes, scales,
                                r.rows, r.K, r.stride, y);
  return r.tiles ? launch_pdl(k_mx_dequantize<false, true>, grid, block, 0, st, codes, scales,
                              r.rows, r.K, r.stride, y)
                 : launch_pdl(k_mx_dequantize<false, false>, grid, block, 0, st, codes, scales,
                              r.rows, r.K, r.stride, y);
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
