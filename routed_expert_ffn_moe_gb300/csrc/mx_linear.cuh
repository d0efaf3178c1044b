// Shared by the two kernels of the MXFP4 product (mx_linear.cu, mx_linear_pair.cu).
#pragma once

#include "mx.h"
#include "tc_common.cuh"

namespace moe {
namespace mxl {

using namespace ptx;
using namespace tc;

constexpr int kStageK = 256;
constexpr uint32_t kRowBytes = kStageK / 2;
constexpr uint32_t kSfBytes = 2 * kMxTile;  // a stage's scales of 128 rows

struct LinParams {
  int T, N, K;
  int mtiles;   // tiles of 128 rows of w
  int splits;   // CTAs of a cluster, along K
  int chunks;   // 128-wide blocks of K
  int64_t x_stride, y_stride, r_stride;
  const uint16_t* x;        // bf16, quantised by the warps
  const uint8_t* x_scales;  // or tiles of scales
  const uint8_t* w_scales;
  const float* bias;
  const uint16_t* residual;
  uint16_t* y;
  int early;  // the kernel ahead is the call's own quantisation of x
  int vec;  // rows of y and of the residual: 8-byte accesses
  int* status;
};

// Bounded wait on an mbarrier phase, as wait_bar, but the clock is first read after 64 tries.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                           int* status) {
  uint64_t t0 = 0;
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63u) == 0) {
      if (*abort_flag) return false;
      const uint64_t t = globaltimer();
      if (t0 == 0) t0 = t;
      if (t - t0 > kWaitLimitNs) {
        record_error(status, MOE_ERR_DEVICE_TIMEOUT);
        *abort_flag = 1;
        return false;
      }
    }
  }
}

// One value of y: the sum, the bias and the residual, rounded once.
__device__ __forceinline__ float with_residual(float v, uint16_t r) {
  return v + __uint_as_float((uint32_t)r << 16);
}

cudaError_t launch_pair(const LinParams& p, const uint8_t* codes, const uint8_t* w,
                        cudaStream_t st);

}  // namespace mxl
}  // namespace moe
