// Interface of the MXFP4 operators: quantisation and back (mx_quant.cu), the product (mx_linear.cu).
#pragma once

#include "internal.h"

namespace moe {

// moe_mx_rows with its defaults filled in
struct MxRows {
  long rows;
  int K;
  bool f32, tiles;
  int64_t stride;
};

// moe_mx_shape with its defaults filled in
struct MxDims {
  int T, N, K;
  bool quantised;  // x is in MXFP4
  int64_t x_stride, y_stride, r_stride;
};

// Scales in tiles: 512 bytes for 128 rows x 128 elements, the chunks of the same rows in a row.
constexpr int kMxTile = 512;
inline __host__ __device__ int mx_chunks(int K) { return (K + 127) / 128; }
inline size_t mx_tile_bytes(long rows, int K) {
  return (size_t)((rows + 127) / 128) * mx_chunks(K) * kMxTile;
}
inline size_t mx_scale_bytes(const MxRows& r) {
  return r.tiles ? mx_tile_bytes(r.rows, r.K) : (size_t)r.rows * (r.K / 32);
}

// workspace of moe_mx_linear: the status word, then x's codes and tiled scales where the call
// quantises them ahead of the product
struct MxWs {
  size_t status, codes, scales, total;
};
inline MxWs mx_ws(const MxDims& d) {
  MxWs w{};
  w.codes = 256;
  w.scales = align_up(w.codes + (d.quantised ? 0 : (size_t)d.T * (d.K / 2)), 256);
  w.total = align_up(w.scales + (d.quantised ? 0 : mx_tile_bytes(d.T, d.K)), 256);
  return w;
}

cudaError_t launch_mx_quantize(const MxRows& r, const void* x, uint8_t* codes, uint8_t* scales,
                               cudaStream_t st);
cudaError_t launch_mx_dequantize(const MxRows& r, const uint8_t* codes, const uint8_t* scales,
                                 void* y, cudaStream_t st);
cudaError_t launch_mx_tile_scales(long rows, int K, const uint8_t* scales, uint8_t* tiles,
                                  cudaStream_t st);
cudaError_t launch_mx_linear(const MxDims& d, const void* x, const uint8_t* x_scales,
                             const uint8_t* w, const uint8_t* w_scales, const float* bias,
                             const uint16_t* residual, uint16_t* y, char* ws, const MxWs& L,
                             cudaStream_t st);

}  // namespace moe
