// The C ABI of the MXFP4 operators (include/moe.h): host-side validation and dispatch.
#include <initializer_list>

#include "capi.h"
#include "mx.h"
#include "ranges.h"

namespace moe {
namespace {

moe_status check_k(int K) {
  if (K < 32 || K > (1 << 17) || K % 32)
    return fail(MOE_ERR_INVALID_ARG, "K=%d not a multiple of 32 in [32, 2^17]", K);
  return MOE_OK;
}

// `given` elements between rows of at least `row`, or the packed rows if 0; offsets fit 63 bits
moe_status take(const char* name, int64_t given, int64_t row, int multiple, int64_t* out) {
  *out = given ? given : row;
  if (*out < row || *out > (int64_t)1 << 36 || *out % multiple)
    return fail(MOE_ERR_INVALID_ARG, "%s=%lld not a multiple of %d of at least %lld elements", name,
                (long long)given, multiple, (long long)row);
  return MOE_OK;
}

moe_status check_rows(const moe_mx_rows* s, MxRows* r) {
  if (!s) return fail(MOE_ERR_INVALID_ARG, "rows is NULL");
  if (s->rows < 0 || s->rows > (1 << 24))
    return fail(MOE_ERR_INVALID_ARG, "rows=%d not in [0, 2^24]", s->rows);
  if (s->dtype != MOE_T_BF16 && s->dtype != MOE_T_F32)
    return fail(MOE_ERR_INVALID_ARG, "dtype=%d: bf16 or fp32 is needed", s->dtype);
  moe_status st = check_k(s->K);
  if (st != MOE_OK) return st;
  r->rows = s->rows;
  r->K = s->K;
  r->f32 = s->dtype == MOE_T_F32;
  r->tiles = s->tiles != 0;
  return take("stride", s->stride, s->K, r->f32 ? 4 : 8, &r->stride);
}

moe_status check_linear(const moe_mx_shape* s, MxDims* d) {
  if (!s) return fail(MOE_ERR_INVALID_ARG, "shape is NULL");
  if (s->T < 0 || s->T > (1 << 24))
    return fail(MOE_ERR_INVALID_ARG, "T=%d not in [0, 2^24]", s->T);
  if (s->N < 1 || s->N > (1 << 20))
    return fail(MOE_ERR_INVALID_ARG, "N=%d not in [1, 2^20]", s->N);
  moe_status st = check_k(s->K);
  if (st != MOE_OK) return st;
  if (s->x_dtype != MOE_T_BF16 && s->x_dtype != MOE_T_MXFP4)
    return fail(MOE_ERR_INVALID_ARG, "x_dtype=%d: bf16 or MXFP4 is needed", s->x_dtype);
  d->T = s->T;
  d->N = s->N;
  d->K = s->K;
  d->quantised = s->x_dtype == MOE_T_MXFP4;
  if (d->quantised && s->x_stride)
    return fail(MOE_ERR_INVALID_ARG, "x_stride=%lld: rows of codes are packed",
                (long long)s->x_stride);
  if ((st = take("x_stride", s->x_stride, s->K, 8, &d->x_stride)) != MOE_OK) return st;
  if ((st = take("y_stride", s->y_stride, s->N, 1, &d->y_stride)) != MOE_OK) return st;
  return take("r_stride", s->r_stride, s->N, 1, &d->r_stride);
}

// An array of the call: absent ones overlap nothing.
struct Array {
  const char* name;
  Runs runs;
  Array(const char* n, const void* p, int64_t bytes) : name(n), runs(p, p ? bytes : 0) {}
  Array(const char* n, const void* p, int64_t rows, int64_t row_bytes, int64_t step)
      : name(n), runs(p, p ? rows : 0, row_bytes, step) {}
};

// Blocks read the inputs while others store: what a call writes lies apart from all else of it.
moe_status apart(const Array& written, std::initializer_list<Array> others) {
  for (const Array& o : others)
    if (overlap(written.runs, o.runs))
      return fail(MOE_ERR_INVALID_ARG, "%s overlaps %s", written.name, o.name);
  return MOE_OK;
}

Array wide_of(const char* name, const void* p, const MxRows& r) {
  const int64_t size = r.f32 ? 4 : 2;
  return Array(name, p, r.rows, r.K * size, r.stride * size);
}
Array codes_of(const char* name, const void* p, int64_t rows, int K) {
  return Array(name, p, rows * (K / 2));
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_mx_scale_bytes(const moe_mx_rows* rows) {
  MxRows r;
  return check_rows(rows, &r) == MOE_OK ? mx_scale_bytes(r) : 0;
}

moe_status moe_mx_quantize(const moe_mx_rows* rows, const void* x, void* codes, void* scales,
                           void* stream) {
  MxRows r;
  moe_status st = check_rows(rows, &r);
  if (st != MOE_OK) return st;
  if (r.rows == 0) return MOE_OK;
  REQUIRE_PTR(x, 16);
  REQUIRE_PTR(codes, 16);
  REQUIRE_PTR(scales, 16);
  if (codes == x || scales == x || codes == scales)
    return fail(MOE_ERR_INVALID_ARG, "x, codes and scales are arrays of their own");
  const Array wide = wide_of("x", x, r), c = codes_of("codes", codes, r.rows, r.K);
  const Array sc("scales", scales, (int64_t)mx_scale_bytes(r));
  if ((st = apart(c, {wide, sc})) != MOE_OK || (st = apart(sc, {wide})) != MOE_OK) return st;
  cudaError_t e = launch_mx_quantize(r, x, static_cast<uint8_t*>(codes),
                                     static_cast<uint8_t*>(scales),
                                     static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : cuda_fail(e, "moe_mx_quantize launch");
}

moe_status moe_mx_dequantize(const moe_mx_rows* rows, const void* codes, const void* scales,
                             void* y, void* stream) {
  MxRows r;
  moe_status st = check_rows(rows, &r);
  if (st != MOE_OK) return st;
  if (r.rows == 0) return MOE_OK;
  REQUIRE_PTR(codes, 16);
  REQUIRE_PTR(scales, 16);
  REQUIRE_PTR(y, 16);
  if (y == codes || y == scales)
    return fail(MOE_ERR_INVALID_ARG, "y is an array of its own");
  if ((st = apart(wide_of("y", y, r), {codes_of("codes", codes, r.rows, r.K),
                                       Array("scales", scales, (int64_t)mx_scale_bytes(r))})) != MOE_OK)
    return st;
  cudaError_t e = launch_mx_dequantize(r, static_cast<const uint8_t*>(codes),
                                       static_cast<const uint8_t*>(scales), y,
                                       static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : cuda_fail(e, "moe_mx_dequantize launch");
}

moe_status moe_mx_tile_scales(const moe_mx_rows* rows, const void* scales, void* tiles,
                              void* stream) {
  MxRows r;
  moe_status st = check_rows(rows, &r);
  if (st != MOE_OK) return st;
  if (r.rows == 0) return MOE_OK;
  REQUIRE_PTR(scales, 16);
  REQUIRE_PTR(tiles, 16);
  if (scales == tiles) return fail(MOE_ERR_INVALID_ARG, "scales and tiles are the same array");
  if ((st = apart(Array("tiles", tiles, (int64_t)mx_tile_bytes(r.rows, r.K)),
                  {Array("scales", scales, r.rows * (r.K / 32))})) != MOE_OK)
    return st;
  cudaError_t e = launch_mx_tile_scales(r.rows, r.K, static_cast<const uint8_t*>(scales),
                                        static_cast<uint8_t*>(tiles),
                                        static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : cuda_fail(e, "moe_mx_tile_scales launch");
}

size_t moe_mx_linear_workspace_size(const moe_mx_shape* shape) {
  MxDims d;
  return check_linear(shape, &d) == MOE_OK ? mx_ws(d).total : 0;
}

moe_status moe_mx_linear(const moe_mx_shape* shape, const void* x, const void* x_scales,
                         const void* w, const void* w_scales, const float* bias,
                         const void* residual, void* y, void* ws, size_t ws_bytes, void* stream) {
  MxDims d;
  moe_status st = check_linear(shape, &d);
  if (st != MOE_OK) return st;
  REQUIRE_PTR(ws, 256);
  const MxWs L = mx_ws(d);
  if (ws_bytes < L.total)
    return fail(MOE_ERR_WORKSPACE, "workspace %zu bytes < %zu required", ws_bytes, L.total);
  if (d.T == 0) return MOE_OK;
  REQUIRE_PTR(x, 16);
  if (d.quantised) REQUIRE_PTR(x_scales, 16);
  if (!d.quantised && x_scales)
    return fail(MOE_ERR_INVALID_ARG, "x_scales must be NULL for a bf16 x");
  REQUIRE_PTR(w, 16);
  REQUIRE_PTR(w_scales, 16);
  REQUIRE_PTR(y, 16);
  if (y == x || y == w) return fail(MOE_ERR_INVALID_ARG, "y is x or w: blocks still read them");
  if (!aligned(bias, 16)) return fail(MOE_ERR_INVALID_ARG, "bias not 16-byte aligned");
  if (!aligned(residual, 16)) return fail(MOE_ERR_INVALID_ARG, "residual not 16-byte aligned");
  if (residual == y && d.r_stride != d.y_stride)
    return fail(MOE_ERR_INVALID_ARG, "residual is y but r_stride=%lld is not y_stride=%lld",
                (long long)d.r_stride, (long long)d.y_stride);
  const Array ax = d.quantised ? codes_of("x", x, d.T, d.K)
                               : Array("x", x, d.T, (int64_t)d.K * 2, d.x_stride * 2);
  const Array axs("x_scales", x_scales, (int64_t)mx_tile_bytes(d.T, d.K));
  const Array aw = codes_of("w", w, d.N, d.K);
  const Array aws("w_scales", w_scales, (int64_t)mx_tile_bytes(d.N, d.K));
  const Array ab("bias", bias, (int64_t)d.N * 4), scratch("ws", ws, (int64_t)L.total);
  const Array ar("residual", residual == y ? nullptr : residual, d.T, (int64_t)d.N * 2, d.r_stride * 2);
  const Array ay("y", y, d.T, (int64_t)d.N * 2, d.y_stride * 2);
  if ((st = apart(ay, {ax, axs, aw, aws, ab, ar, scratch})) != MOE_OK ||
      (st = apart(scratch, {ax, axs, aw, aws, ab, ar})) != MOE_OK)
    return st;
  cudaError_t e = launch_mx_linear(
      d, x, static_cast<const uint8_t*>(x_scales), static_cast<const uint8_t*>(w),
      static_cast<const uint8_t*>(w_scales), bias, static_cast<const uint16_t*>(residual),
      static_cast<uint16_t*>(y), static_cast<char*>(ws), L, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : cuda_fail(e, "moe_mx_linear launch");
}

}  // extern "C"
