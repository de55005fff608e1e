// The forward of the residual operator (residual.hip has the formulas), shared by its two outputs:
// rows of the layer's type, and rows in 8 bits with scales (residual_mx.hip).
#pragma once

#include <algorithm>

#include "dropout.h"
#include "launch.h"
#include "mx.h"
#include "residual.h"
#include "row8.h"

namespace moe {

namespace {

// ------------------------------------------------------------------ forward
// Mean and 1 / deviation of a row held as float32 (zeros past its end, which `live` keeps out of a
// layer norm's squares).
template <int TPR, int CH>
__device__ __forceinline__ void row_stats(const float (&u)[CH][8], const bool (&live)[CH],
                                          bool layer, float inv_h, float eps, RowSum<TPR>& sum,
                                          float& mean, float& rstd) {
  mean = 0.f;
  if (layer) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) s += u[i][j];
    mean = sum(s, 0.f).x * inv_h;
  }
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const float m = live[i] ? mean : 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float c = u[i][j] - m;
      q = fmaf(c, c, q);
    }
  }
  rstd = 1.0f / sqrtf(sum(q, 0.f).x * inv_h + eps);
}

// MX: x' also (or only, x_out null) in 8 bits with scales.
//
// TPR threads a row, in CH chunks of 8 elements a thread; each takes every so many-th row, with
// the vectors along H in registers over the rows and the next row in flight while one is reduced.
// A row is read once and h', x' are written once. A thread reads all of its h and y before it
// writes anything of that row, so h' may be h. Bound by HBM (8192 x 2880 bf16 with one norm:
// 37.8 us, 5.0 TB/s, where a large copy takes 37; 16384 x 2048 fp16 with both norms, a gate and
// dropout: 55.8 us, a copy 53; one row: 2.6 us).
template <typename Elem, int TPR, int CH, int GATE, bool MX>
__global__ __launch_bounds__(row_block<TPR>()) void residual_fwd_kernel(ResidualArgs p) {
  constexpr int BLOCK = row_block<TPR>(), R = BLOCK / TPR;
  __shared__ float slots[2][2 * (TPR / kWave)];
  const int lane = row_lane<TPR>();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * R + row_in_block<TPR>();
  const int64_t stride = static_cast<int64_t>(gridDim.x) * R;
  RowSum<TPR> sum{slots, 0};
  const int cpr = p.H / 8, rb = p.H * static_cast<int>(sizeof(Elem));
  const bool post = p.post != MOE_NORM_NONE, pre = p.pre != MOE_NORM_NONE;
  const bool dropout = p.drop.thr != 0;
  const DropKey key = drop_key(p.drop);

  Row8<Elem> nh[CH], ny[CH];
  auto fetch = [&](int64_t row) __attribute__((always_inline)) {
    const auto bh = row_buf(p.h, row, rb, row < p.T), by = row_buf(p.y, row, rb, row < p.T);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      ny[i].load(by, lane + i * TPR);
      nh[i].load(bh, lane + i * TPR);
    }
  };
  fetch(first);
  // as they are applied: shift + w, and the gate's value; 0 past the row
  bool live[CH];
  float wpost[CH][8], bpost[CH][8], wpre[CH][8], bpre[CH][8], gch[CH][8];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    live[i] = lane + i * TPR < cpr;
    auto vector = [&](const void* v, float add, float (&out)[8]) {
      Row8<Elem> r;
      r.load(row_buf(v, 0, rb), lane + i * TPR);
      r.get(out);
#pragma unroll
      for (int j = 0; j < 8; ++j) out[j] = live[i] ? out[j] + add : 0.f;
    };
    vector(p.w_post, p.shift, wpost[i]);
    vector(p.b_post, 0.f, bpost[i]);
    vector(p.w_pre, p.shift, wpre[i]);
    vector(p.b_pre, 0.f, bpre[i]);
    if (GATE == MOE_GATE_CHANNEL) {
      vector(p.gate, 0.f, gch[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) gch[i][j] = gate_value(gch[i][j], p.gate_sigmoid);
    }
  }

  for (int64_t row = first; row < p.T; row += stride) {
    Row8<Elem> rh[CH], ry[CH], rg[CH];
    if (GATE == MOE_GATE_FULL) {
      const auto bg = row_buf(p.gate, row, rb);
#pragma unroll
      for (int i = 0; i < CH; ++i) rg[i].load(bg, lane + i * TPR);
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      rh[i] = nh[i];
      ry[i] = ny[i];
    }
    fetch(row + stride);
    // the mask needs nothing from memory: drawn while the row arrives
    uint4 rnd[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      rnd[i] = make_uint4(0, 0, 0, 0);
      if (dropout) rnd[i] = philox(key, static_cast<uint64_t>(row * cpr + lane + i * TPR));
    }
    float gt = 1.f;
    if (GATE == MOE_GATE_TOKEN)
      gt = gate_value(to_f32<Elem>(static_cast<const Elem*>(p.gate)[row]), p.gate_sigmoid);
    float4 st = make_float4(0.f, 0.f, 0.f, 0.f);
    float u[CH][8];
#pragma unroll
    for (int i = 0; i < CH; ++i) ry[i].get(u[i]);
    if (post) {
      row_stats<TPR, CH>(u, live, p.post == MOE_NORM_LAYER, p.inv_h, p.eps, sum, st.x, st.y);
      const float off = -st.x * st.y;
#pragma unroll
      for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          u[i][j] = fmaf(fmaf(u[i][j], st.y, off), wpost[i][j], bpost[i][j]);
    }
    const auto bho = row_buf(p.h_out, row, rb);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      float h[8];
      if (GATE == MOE_GATE_FULL) {
        float g[8];
        rg[i].get(g);
#pragma unroll
        for (int j = 0; j < 8; ++j) u[i][j] *= gate_value(g[j], p.gate_sigmoid);
      }
      if (GATE == MOE_GATE_CHANNEL) {
#pragma unroll
        for (int j = 0; j < 8; ++j) u[i][j] *= gch[i][j];
      }
      const float k = GATE == MOE_GATE_TOKEN ? p.alpha * gt : p.alpha;
      // scaled before the sum rather than through k: the result is the one of moe_dropout and an
      // add, bit for bit
      if (dropout) {
#pragma unroll
        for (int j = 0; j < 8; ++j) u[i][j] = drop(p.drop, rnd[i], j, u[i][j]);
      }
      rh[i].get(h);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] = fmaf(k, u[i][j], h[j]);
      rh[i].set(h);
      rh[i].store(bho, lane + i * TPR);
      rh[i].get(u[i]);  // h' as it is stored
    }
    if (pre) {
      row_stats<TPR, CH>(u, live, p.pre == MOE_NORM_LAYER, p.inv_h, p.eps, sum, st.z, st.w);
      const float off = -st.z * st.w;
      const auto bxo = row_buf(p.x_out, row, rb);
#pragma unroll
      for (int i = 0; i < CH; ++i) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          u[i][j] = fmaf(fmaf(u[i][j], st.w, off), wpre[i][j], bpre[i][j]);
        Row8<Elem> o;
        o.set(u[i]);
        o.store(bxo, lane + i * TPR);
        if constexpr (MX) {
          // from the value as x_out holds it: the bits of this call and of the norm followed by
          // moe_mx_quantize are the same. Lanes past the row write the scales that fill it up, 0.
          o.get(u[i]);
          const uint32_t sc = live[i] ? mx_scale_of<MOE_MX_FP8>(mx_block_amax(u[i])) : 0u;
          const uint2 q = mx_encode8<MOE_MX_FP8>(u[i], sc);
          typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
          const int at = lane + i * TPR;
          __builtin_amdgcn_raw_buffer_store_b64(u32x2{q.x, q.y}, row_buf(p.codes, row, p.H), 8 * at,
                                                0, 0);
          const int scols = static_cast<int>(mx_scale_cols(p.H));
          __builtin_amdgcn_raw_buffer_store_b8(static_cast<uint8_t>(sc),
                                               row_buf(p.scales, row, scols),
                                               (at & 3) == 0 ? at >> 2 : scols, 0, 0);
        }
      }
    }
    if (lane == 0 && p.stats) p.stats[row] = st;
  }
}

template <bool MX>
hipError_t launch_residual_rows(int dtype, const ResidualArgs& a, hipStream_t s) {
  return by_type(dtype, [&](auto tag) {
    return by_row_width(a.H, [&](auto tpr, auto ch) {
      typedef decltype(tag) Elem;
      constexpr int TPR = decltype(tpr)::value, CH = decltype(ch)::value;
      constexpr int BLOCK = row_block<TPR>(), R = BLOCK / TPR;
      // as many blocks as a CU holds by registers, over 256 CUs: one round, no tail
      const int64_t rows = (static_cast<int64_t>(a.T) + R - 1) / R;
      const int64_t blocks = 256 * std::max(1, 1024 / BLOCK);
      auto* kern = a.gate_kind == MOE_GATE_CHANNEL ? residual_fwd_kernel<Elem, TPR, CH, MOE_GATE_CHANNEL, MX>
                   : a.gate_kind == MOE_GATE_TOKEN ? residual_fwd_kernel<Elem, TPR, CH, MOE_GATE_TOKEN, MX>
                   : a.gate_kind == MOE_GATE_FULL  ? residual_fwd_kernel<Elem, TPR, CH, MOE_GATE_FULL, MX>
                                                   : residual_fwd_kernel<Elem, TPR, CH, MOE_GATE_NONE, MX>;
      hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(std::min(rows, blocks))),
                         dim3(BLOCK), 0, s, a);
      return hipGetLastError();
    });
  });
}

}  // namespace

}  // namespace moe
