// Microscaled formats: 32 consecutive elements of a row share one scale 2^(s - 127), s a byte (E8M0,
// 255: NaN), and are held as E2M1 (4 bits, two a byte, the first in the low half) or E4M3 (8 bits).
//
//   s = max(0, floor(log2(amax)) + 127 - top)     top: exponent of the format's largest value, 2 or 8
//   code = the nearest value to x / 2^(s - 127), ties to an even code, at most 6 or 448
//
// A block of zeros has s = 0. An infinity or NaN among the 32 makes s = 255: the block reads as NaN.
#pragma once

#include "device_common.h"
#include "moe_lora.h"
#include "row8.h"

namespace moe {

// scale bytes a row, whole 16-byte pieces (512 elements each); those past the last block are 0
__host__ __device__ __forceinline__ int64_t mx_scale_cols(int64_t cols) {
  return (cols + 511) / 512 * 16;
}
__host__ __device__ __forceinline__ int64_t mx_code_bytes(int fmt, int64_t n) {
  return fmt == MOE_MX_FP4 ? n / 2 : n;
}

// The scale of a block whose largest magnitude is the float with these bits.
template <int FMT>
__device__ __forceinline__ uint32_t mx_scale_of(uint32_t amax_bits) {
  constexpr uint32_t top = FMT == MOE_MX_FP4 ? 2 : 8;
  const uint32_t e = amax_bits >> 23;  // 0 for zero and what is below float32's normal range
  return e == 255 ? 255u : (e > top ? e - top : 0u);
}

// The largest magnitude's bits over the four lanes (a quad) that hold a block, 8 elements each.
// Magnitudes order as their bits do, and NaN comes out on top of them.
__device__ __forceinline__ uint32_t mx_block_amax(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
  m = max(m, static_cast<uint32_t>(dpp_i32<kDppSwap1>(static_cast<int>(m))));
  m = max(m, static_cast<uint32_t>(dpp_i32<kDppSwap2>(static_cast<int>(m))));
  return m;
}

// Eight elements as codes of the scale s: 8 bytes of E4M3 or 4 of E2M1 (the other word 0). The
// conversions divide by the power of two whose exponent bits they are given and round to nearest
// even; the one to 4 bits stops at 6 by itself, the one to 8 bits would give NaN above 464.
template <int FMT>
__device__ __forceinline__ uint2 mx_encode8(const float (&v)[8], uint32_t s) {
  uint2 r = make_uint2(0, 0);
  if (s == 255) return r;
  const float scale = __uint_as_float(s << 23);
  if constexpr (FMT == MOE_MX_FP4) {
    r.x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r.x, v[0], v[1], scale, 0);
    r.x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r.x, v[2], v[3], scale, 1);
    r.x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r.x, v[4], v[5], scale, 2);
    r.x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r.x, v[6], v[7], scale, 3);
  } else {
    typedef short s16x2 __attribute__((ext_vector_type(2)));
    // 448 2^(s - 127) = 1.75 2^(s - 119), in range since s <= 246
    const float most = __uint_as_float(((s + 8) << 23) | 0x600000u);
    float c[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = __builtin_amdgcn_fmed3f(v[j], most, -most);
    s16x2 a = {0, 0}, b = {0, 0};
    a = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(a, c[0], c[1], scale, false);
    a = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(a, c[2], c[3], scale, true);
    b = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(b, c[4], c[5], scale, false);
    b = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(b, c[6], c[7], scale, true);
    r.x = __builtin_bit_cast(uint32_t, a);
    r.y = __builtin_bit_cast(uint32_t, b);
  }
  return r;
}

// Eight values of codes with the scale s.
template <int FMT>
__device__ __forceinline__ void mx_decode8(uint2 c, uint32_t s, float (&v)[8]) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  // 2^-127 is below float32's normal range
  const float scale = s == 255 ? __uint_as_float(0x7fc00000u)
                               : s == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(s << 23);
  f32x2 p[4];
  if constexpr (FMT == MOE_MX_FP4) {
    p[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c.x, 1.0f, 0);
    p[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c.x, 1.0f, 1);
    p[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c.x, 1.0f, 2);
    p[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c.x, 1.0f, 3);
  } else {
    p[0] = __builtin_amdgcn_cvt_pk_f32_fp8(c.x, false);
    p[1] = __builtin_amdgcn_cvt_pk_f32_fp8(c.x, true);
    p[2] = __builtin_amdgcn_cvt_pk_f32_fp8(c.y, false);
    p[3] = __builtin_amdgcn_cvt_pk_f32_fp8(c.y, true);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = p[j][0] * scale;
    v[2 * j + 1] = p[j][1] * scale;
  }
}

// Calls go with the format as a constant.
template <typename F>
hipError_t by_format(int fmt, F&& go) {
  if (fmt == MOE_MX_FP4) return go(std::integral_constant<int, MOE_MX_FP4>());
  return go(std::integral_constant<int, MOE_MX_FP8>());
}

}  // namespace moe
