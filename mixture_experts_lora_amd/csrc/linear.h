// Epilogue of the linear operator: y = residual + dropout(act(z)), z = x w^T + bias, on eight
// consecutive columns of a row, shared by its GEMMs, its few-token kernel and its split-K sum.
#pragma once

#include <type_traits>

#include "dropout.h"
#include "row8.h"

namespace moe {

// exp2 and reciprocal of the hardware, each within 1 ulp (sigmoidf_). The tanh form of gelu uses
// (1 + tanh u) / 2 = sigmoid(2u), which also avoids the sum's cancellation for negative z.
constexpr float kGeluC = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

// Phi(z), and e = exp(-z^2 / 2).
//
// float: erfc(-z / sqrt 2) / 2, which keeps its relative accuracy where Phi is small, by the math
// library; the float32 products take far longer than its about eighty instructions.
//
// 16-bit types: Abramowitz and Stegun 7.1.26 (erfc as a polynomial in t = 1 / (1 + p x) times
// exp(-x^2), within 1.5e-7), a dozen instructions that the slope's exponential is part of: the
// library's erf and exponential bound the kernel that forms dz (8192 x 2880, gelu: 43 us, with the
// polynomial 27.6). Relative to Phi it is off by 8e-7 at most above -1, 5.3e-5 above -3, 4.7e-4
// above -4 and 3.6e-3 above -6, so the output's rounding is the larger error (bf16: 3.9e-3; fp16:
// 4.9e-4, and coarser below 6e-5, which |z Phi(z)| reaches at -4.2) until |z Phi(z)| is below 6e-9.
template <typename Elem>
__device__ __forceinline__ float gelu_phi(float z, float& e) {
  if constexpr (std::is_same_v<Elem, float>) {
    e = expf(-0.5f * z * z);
    return 0.5f * erfcf(z * -0.7071067811865476f);
  }
  const float x = fabsf(z) * 0.7071067811865476f;
  e = __expf(-x * x);
  const float t = __builtin_amdgcn_rcpf(fmaf(0.3275911f, x, 1.f));
  float q = fmaf(1.061405429f, t, -1.453152027f);
  q = fmaf(q, t, 1.421413741f);
  q = fmaf(q, t, -0.284496736f);
  q = fmaf(q, t, 0.254829592f);
  const float half_erfc = 0.5f * q * t * e;
  return z < 0.f ? half_erfc : 1.f - half_erfc;
}

template <typename Elem>
__device__ __forceinline__ float act_value(float z, int act) {
  switch (act) {
    case MOE_ACT_RELU: return z < 0.f ? 0.f : z;
    case MOE_ACT_SILU: return z * sigmoidf_(z);
    case MOE_ACT_GELU: {
      float e;
      return z * gelu_phi<Elem>(z, e);
    }
    case MOE_ACT_GELU_TANH: return z * sigmoidf_(2.f * kGeluC * (z + kGeluA * z * z * z));
    default: return z;
  }
}

// Slopes. Their terms that grow with z take it clamped to where its other factor is 0 or 1 already, so
// that the limits 0 and 1 come out however large z is (z^2 overflows from 2e19 on).
template <typename Elem>
__device__ __forceinline__ float act_slope(float z, int act) {
  const float c = fminf(fmaxf(z, -128.f), 128.f);
  switch (act) {
    case MOE_ACT_RELU: return z > 0.f ? 1.f : 0.f;
    case MOE_ACT_SILU: {
      const float s = sigmoidf_(z);
      return s * (1.f + c * (1.f - s));
    }
    case MOE_ACT_GELU: {  // Phi(z) + z phi(z)
      float e;
      const float phi = gelu_phi<Elem>(z, e);
      return fmaf(c * 0.3989422804014327f, e, phi);
    }
    case MOE_ACT_GELU_TANH: {
      const float s = sigmoidf_(2.f * kGeluC * (z + kGeluA * z * z * z));
      return s + 2.f * kGeluC * c * s * (1.f - s) * (1.f + 3.f * kGeluA * c * c);
    }
    default: return 1.f;
  }
}

// v: the product's columns col .. col + 7 of `row`; ncols (a multiple of 8) is y's row length; bias,
// res: the bias's and the residual's elements there (zeros without one).
template <typename Elem>
__device__ __forceinline__ void linear_finish8(const LinearEpi& q, const DropKey& key, int64_t row,
                                               int col, int ncols, const Row8<Elem>& bias,
                                               const Row8<Elem>& res, float (&v)[8]) {
  const int64_t at = row * ncols + col;
  Row8<Elem> r;
  float f[8];
  bias.get(f);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = fmaf(v[j], q.scale, f[j]);
  if (q.pre) {
    r.set(v);
    r.store(static_cast<Elem*>(q.pre) + at);
  }
  if (q.act != MOE_ACT_NONE) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = act_value<Elem>(v[j], q.act);
  }
  if (q.drop.thr) {
    const uint4 rnd = philox(key, static_cast<uint64_t>(at) / 8);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = drop(q.drop, rnd, j, v[j]);
  }
  res.get(f);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] += f[j];
  r.set(v);
  r.store(static_cast<Elem*>(q.y) + at);
}

// The same with the bias and the residual loaded here.
template <typename Elem>
__device__ __forceinline__ void linear_finish8(const LinearEpi& q, int64_t row, int col, int ncols,
                                               float (&v)[8]) {
  Row8<Elem> bias, res;
  bias.zero();
  res.zero();
  if (q.bias) bias.load(static_cast<const Elem*>(q.bias) + col);
  if (q.residual) res.load(static_cast<const Elem*>(q.residual) + row * ncols + col);
  linear_finish8<Elem>(q, drop_key(q.drop), row, col, ncols, bias, res, v);
}

}  // namespace moe
