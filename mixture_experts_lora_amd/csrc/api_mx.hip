// C ABI of the microscaled formats: argument checks and launches (include/moe_lora.h has the
// contract of every entry point).
#include <algorithm>
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

moe_status check_mx_linear(const moe_mx_linear_shape* s) {
  if (!s) return fail(MOE_ERR_INVALID_ARG, "null shape");
  if (s->T < 1 || s->K < 1 || s->N < 1 || s->k < 1)
    return fail(MOE_ERR_INVALID_ARG, "T, K, N and k must be >= 1");
  if (s->E < 0 || s->E > 1024) return fail(MOE_ERR_INVALID_ARG, "E must be in [0, 1024]");
  if (s->E == 0 && (s->k != 1 || s->gather))
    return fail(MOE_ERR_INVALID_ARG, "one weight matrix takes k = 1 and no gather");
  if (s->E > 0 && (s->k > s->E || s->k > 32))
    return fail(MOE_ERR_INVALID_ARG, "k must be in [1, min(E, 32)]");
  if (s->a_format != MOE_MX_FP8 && s->a_format != MOE_MX_FP4)
    return fail(MOE_ERR_INVALID_ARG, "unknown microscaled format " + std::to_string(s->a_format));
  if (s->out != MOE_BF16 && s->out != MOE_F16 && s->out != MOE_MX_OUT_FP8)
    return fail(MOE_ERR_INVALID_ARG, "unknown output " + std::to_string(s->out));
  if (s->K % 32 != 0) return fail(MOE_ERR_UNSUPPORTED, "K must be a multiple of 32");
  const int unit = s->out == MOE_MX_OUT_FP8 ? 32 : 8;
  if (s->N % unit != 0)
    return fail(MOE_ERR_UNSUPPORTED, "N must be a multiple of " + std::to_string(unit));
  if (s->K > (1 << 20) || s->N > (1 << 20))
    return fail(MOE_ERR_UNSUPPORTED, "K or N > 2^20 is not supported");
  if (int64_t(s->T) * s->k >= (int64_t(1) << 31))
    return fail(MOE_ERR_INVALID_ARG, "T*k must be < 2^31");
  if (int64_t(s->T) * s->k > (int64_t(1) << 34) / std::max(s->K, s->N))
    return fail(MOE_ERR_INVALID_ARG, "activations of more than 2^34 elements");
  // 32-bit buffer offsets into a matrix, and into gathered rows
  if (int64_t(s->N) * (s->swiglu ? 2 : 1) * (s->K / 2) >= (int64_t(1) << 31))
    return fail(MOE_ERR_INVALID_ARG, "the codes of a weight matrix must be smaller than 2 GiB");
  if (s->gather && moe::mx_code_bytes(s->a_format, int64_t(s->T) * s->K) >= (int64_t(1) << 31))
    return fail(MOE_ERR_INVALID_ARG, "the codes of a gathered a must be smaller than 2 GiB");
  // a grid holds fewer than 2^32 threads: tiles of 64 rows and 128 weight rows at 256 each, with one
  // tile that is not full for every expert (larger tiles are taken only for far fewer)
  const int64_t M = int64_t(s->T) * s->k, cols = s->swiglu ? 64 : 128;
  if ((M / 64 + std::max<int64_t>(1, std::min<int64_t>(s->E, M))) * ((s->N + cols - 1) / cols) >= (1 << 24))
    return fail(MOE_ERR_UNSUPPORTED, "more tiles of the experts than a grid holds");
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

moe_status moe_mx_linear_workspace_bytes(const moe_mx_linear_shape* shape, size_t* ws) {
  moe_status st = check_mx_linear(shape);
  if (st != MOE_OK) return st;
  CHECK_PTR(ws);
  *ws = 0;
  return MOE_OK;
}

moe_status moe_mx_linear(const moe_mx_linear_shape* shape, const void* a, const uint8_t* a_scales,
                         const int32_t* rows, const int32_t* offsets, const void* w,
                         const uint8_t* w_scales, void* y, uint8_t* y_scales, void*, size_t,
                         void* stream) {
  moe_status st = check_mx_linear(shape);
  if (st != MOE_OK) return st;
  const moe_mx_linear_shape& s = *shape;
  const bool mx = s.out == MOE_MX_OUT_FP8;
  CHECK_PTR(a);
  CHECK_PTR(a_scales);
  if (s.gather) CHECK_PTR(rows);
  if (s.E > 0) CHECK_PTR(offsets);
  CHECK_PTR(w);
  CHECK_PTR(w_scales);
  CHECK_PTR(y);
  if (mx) CHECK_PTR(y_scales);
  else if (y_scales) return fail(MOE_ERR_INVALID_ARG, "y_scales without an 8-bit output");
  CHECK_ROWS(a);
  CHECK_ROWS(a_scales);
  CHECK_ROWS(w);
  CHECK_ROWS(w_scales);
  CHECK_ROWS(y);
  CHECK_ROWS(y_scales);
  if ((s.gather && (reinterpret_cast<uintptr_t>(rows) & 3)) ||
      (s.E > 0 && (reinterpret_cast<uintptr_t>(offsets) & 3)))
    return fail(MOE_ERR_INVALID_ARG, "rows or offsets do not start on a 4-byte boundary");
  const int64_t M = int64_t(s.T) * s.k, ar = s.gather ? s.T : M, sk = moe::mx_scale_cols(s.K);
  const int64_t wr = int64_t(s.N) * (s.swiglu ? 2 : 1) * (s.E > 0 ? s.E : 1);
  st = check_ranges(
      {{y, M * s.N * (mx ? 1 : 2), "y"}, {y_scales, M * moe::mx_scale_cols(s.N), "y_scales"}},
      {{a, moe::mx_code_bytes(s.a_format, ar * s.K), "a"}, {a_scales, ar * sk, "a_scales"},
       {w, wr * (s.K / 2), "w"}, {w_scales, wr * sk, "w_scales"},
       {s.gather ? rows : nullptr, M * 4, "rows"},
       {s.E > 0 ? offsets : nullptr, (int64_t(s.E) + 1) * 4, "offsets"}});
  if (st != MOE_OK) return st;
  hipError_t e = moe::launch_mx_linear(s, a, a_scales, rows, offsets, w, w_scales, y, y_scales,
                                       as_stream(stream), moe::active_timer());
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_mx_linear");
}

}  // extern "C"
