// C ABI of the microscaled formats: argument checks and launches (include/moe_lora.h has the
// contract of every entry point).
#include <string>

#include "api_check.h"
#include "launch.h"
#include "mx.h"

using namespace moe::check;
using moe::fail;

namespace {

moe_status check_mx(int32_t format, int32_t dtype, int64_t rows, int32_t cols) {
  if (format != MOE_MX_FP8 && format != MOE_MX_FP4)
    return fail(MOE_ERR_INVALID_ARG, "unknown microscaled format " + std::to_string(format));
  if (!known_dtype(dtype)) return fail(MOE_ERR_INVALID_ARG, "unknown dtype");
  if (rows < 0) return fail(MOE_ERR_INVALID_ARG, "rows < 0");
  if (cols < 1 || cols % 32 != 0)
    return fail(MOE_ERR_UNSUPPORTED, "cols must be a positive multiple of 32");
  if (rows >= (int64_t(1) << 34) / cols)
    return fail(MOE_ERR_INVALID_ARG, "2^34 elements or more");
  return MOE_OK;
}

}  // namespace

extern "C" {

int64_t moe_mx_scale_cols(int64_t cols) { return cols > 0 ? moe::mx_scale_cols(cols) : 0; }

moe_status moe_mx_quantize(int32_t format, int32_t dtype, int64_t rows, int32_t cols,
                           const void* src, void* codes, uint8_t* scales, void* stream) {
  moe_status st = check_mx(format, dtype, rows, cols);
  if (st != MOE_OK || rows == 0) return st;
  CHECK_PTR(src);
  CHECK_PTR(codes);
  CHECK_PTR(scales);
  CHECK_ROWS(src);
  CHECK_ROWS(codes);
  CHECK_ROWS(scales);
  const int64_t n = rows * cols;
  st = check_ranges({{codes, moe::mx_code_bytes(format, n), "codes"},
                     {scales, rows * moe::mx_scale_cols(cols), "scales"}},
                    {{src, n * esize(dtype), "src"}});
  if (st != MOE_OK) return st;
  hipError_t e = moe::launch_mx_quantize(format, dtype, rows, cols, src, codes, scales,
                                         as_stream(stream), moe::active_timer());
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_mx_quantize");
}

moe_status moe_mx_dequantize(int32_t format, int32_t dtype, int64_t rows, int32_t cols,
                             const void* codes, const uint8_t* scales, void* dst, void* stream) {
  moe_status st = check_mx(format, dtype, rows, cols);
  if (st != MOE_OK || rows == 0) return st;
  CHECK_PTR(codes);
  CHECK_PTR(scales);
  CHECK_PTR(dst);
  CHECK_ROWS(codes);
  CHECK_ROWS(scales);
  CHECK_ROWS(dst);
  const int64_t n = rows * cols;
  st = check_ranges({{dst, n * esize(dtype), "dst"}},
                    {{codes, moe::mx_code_bytes(format, n), "codes"},
                     {scales, rows * moe::mx_scale_cols(cols), "scales"}});
  if (st != MOE_OK) return st;
  hipError_t e = moe::launch_mx_dequantize(format, dtype, rows, cols, codes, scales, dst,
                                           as_stream(stream), moe::active_timer());
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_mx_dequantize");
}

}  // extern "C"
