// Epilogue of the linear operator: y = residual + dropout(act(z)), z = x w^T + bias, on eight
// consecutive columns of a row, shared by its GEMMs, its few-token kernel and its split-K sum.
#pragma once

#include "dropout.h"
#include "row8.h"

namespace moe {

// exp2 and reciprocal of the hardware, each within 1 ulp (sigmoidf_). The tanh form of gelu uses
// (1 + tanh u) / 2 = sigmoid(2u), which also avoids the sum's cancellation for negative z.
constexpr float kGeluC = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

__device__ __forceinline__ float act_value(float z, int act) {
  switch (act) {
    case MOE_ACT_RELU: return z < 0.f ? 0.f : z;
    case MOE_ACT_SILU: return z * sigmoidf_(z);
    case MOE_ACT_GELU: return 0.5f * z * (1.f + erff(z * 0.7071067811865476f));
    case MOE_ACT_GELU_TANH: return z * sigmoidf_(2.f * kGeluC * (z + kGeluA * z * z * z));
    default: return z;
  }
}

__device__ __forceinline__ float act_slope(float z, int act) {
  switch (act) {
    case MOE_ACT_RELU: return z > 0.f ? 1.f : 0.f;
    case MOE_ACT_SILU: {
      const float s = sigmoidf_(z);
      return s * (1.f + z * (1.f - s));
    }
    case MOE_ACT_GELU:  // Phi(z) + z phi(z)
      return 0.5f * (1.f + erff(z * 0.7071067811865476f)) +
             z * 0.3989422804014327f * __expf(-0.5f * z * z);
    case MOE_ACT_GELU_TANH: {
      const float s = sigmoidf_(2.f * kGeluC * (z + kGeluA * z * z * z));
      return s + 2.f * kGeluC * z * s * (1.f - s) * (1.f + 3.f * kGeluA * z * z);
    }
    default: return 1.f;
  }
}

// v: the product's columns col .. col + 7 of `row`; ncols (a multiple of 8) is y's row length.
template <typename Elem>
__device__ __forceinline__ void linear_finish8(const LinearEpi& q, int64_t row, int col, int ncols,
                                               float (&v)[8]) {
  const int64_t at = row * ncols + col;
  Row8<Elem> r;
  float f[8];
  if (q.bias) {
    r.load(static_cast<const Elem*>(q.bias) + col);
    r.get(f);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += f[j];
  }
  if (q.pre) {
    r.set(v);
    r.store(static_cast<Elem*>(q.pre) + at);
  }
  if (q.act != MOE_ACT_NONE) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = act_value(v[j], q.act);
  }
  if (q.drop.thr) {
    const uint4 rnd = drop_words(q.drop, drop_key(q.drop), static_cast<uint64_t>(at) / 8);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = drop(q.drop, rnd, j, v[j]);
  }
  if (q.residual) {
    r.load(static_cast<const Elem*>(q.residual) + at);
    r.get(f);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += f[j];
  }
  r.set(v);
  r.store(static_cast<Elem*>(q.y) + at);
}

}  // namespace moe
