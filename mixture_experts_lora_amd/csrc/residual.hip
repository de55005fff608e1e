// The residual stream around a block: element-wise dropout, and the fused residual operator
//
//   forward   v  = post(y)                     post, pre: none, RMS norm or layer norm
//             h' = h + alpha g drop(v)         g: 1, or a gate per channel, token or element
//             x' = pre(h')                     h' as it is stored (rounded to the layer dtype)
//   backward  D  = dh' + J_pre(h')^T dx'       the gradient at h'; dh = D
//             dg = alpha drop(v) D             summed over the gate's broadcast axis
//             e  = alpha g drop(D)             the gradient at v, under the same mask
//             dy = J_post(y)^T e
//
// A norm is n(u) = (shift + w) uhat + b with uhat = (u - mean) rstd (mean = 0 for RMS, b = 0 and
// none for RMS), rstd = 1 / sqrt(mean((u - mean)^2) + eps), and with d = (shift + w) dn its input
// gradient is rstd (d - mean(d) - uhat mean(d uhat)) (no mean(d) for RMS); dw = sum_t dn uhat,
// db = sum_t dn.
//
// Both directions are bound by HBM: they move each row once and hold it in registers between the
// reductions. All sums, means and the stored statistics are float32. A variance is the mean
// square about the mean already found (the row is at hand), not a difference of moments.
#include <algorithm>
#include <type_traits>

#include "dropout.h"
#include "launch.h"
#include "residual.h"
#include "row8.h"

namespace moe {

namespace {

// ------------------------------------------------------------------ element-wise dropout
// One thread per 8 elements (one counter); VEC: both pointers on a 16-byte boundary. src and dst
// may be the same buffer: a thread reads its elements before it writes them. Bound by HBM: the
// generator's twenty multiplies serve 16 bytes read and 16 written (65536 x 2880 bf16: 123.5 us,
// 6.1 TB/s, part of it from the last-level cache; 300 x 584: 2.4 us).
template <typename Elem, bool VEC>
__global__ __launch_bounds__(256) void dropout_kernel(const Elem* src, Elem* dst, int64_t c0,
                                                      int64_t n, DropArgs d) {
  const int64_t c = c0 + static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, i = c * 8;
  if (i >= n) return;
  const DropKey key = drop_key(d);
  Row8<Elem> r;
  const bool whole = VEC && i + 8 <= n;
  if (whole) r.load(src + i);
  const uint4 rnd = drop_words(d, key, static_cast<uint64_t>(c));
  if (whole) {
    float v[8];
    r.get(v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = drop(d, rnd, j, v[j]);
    r.set(v);
    r.store(dst + i);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < n) dst[i + j] = from_f32<Elem>(drop(d, rnd, j, to_f32<Elem>(src[i + j])));
  }
}

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

// TPR threads a row, in CH chunks of 8 elements a thread; each takes every so many-th row, with
// the vectors along H in registers over the rows and the next row in flight while one is reduced.
// A row is read once and h', x' are written once. A thread reads all of its h and y before it
// writes anything of that row, so h' may be h. Bound by HBM (8192 x 2880 bf16 with one norm:
// 37.8 us, 5.0 TB/s, where a large copy takes 37; 16384 x 2048 fp16 with both norms, a gate and
// dropout: 55.8 us, a copy 53; one row: 2.6 us).
template <typename Elem, int TPR, int CH, int GATE>
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
      }
    }
    if (lane == 0 && p.stats) p.stats[row] = st;
  }
}

}  // namespace

hipError_t launch_dropout(int dtype, int64_t n, const DropArgs& d, const void* src, void* dst,
                          hipStream_t s, KernelTimer* tm) {
  TimedScope ts(tm, MOE_K_DROPOUT, s);
  const bool vec = ((reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst)) & 15) == 0;
  const int64_t chunks = (n + 7) / 8;
  return by_type(dtype, [&](auto tag) {
    using Elem = decltype(tag);
    auto* kern = vec ? dropout_kernel<Elem, true> : dropout_kernel<Elem, false>;
    // a grid has fewer than 2^32 threads
    constexpr int64_t kMost = int64_t(1) << 31;
    for (int64_t c0 = 0; c0 < chunks; c0 += kMost) {
      const dim3 grid(static_cast<unsigned>((std::min(kMost, chunks - c0) + 255) / 256));
      hipLaunchKernelGGL(kern, grid, dim3(256), 0, s, static_cast<const Elem*>(src),
                         static_cast<Elem*>(dst), c0, n, d);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  });
}

hipError_t launch_residual_fwd(int dtype, const ResidualArgs& a, hipStream_t s, KernelTimer* tm) {
  TimedScope ts(tm, MOE_K_RESIDUAL_NORM, s);
  return by_type(dtype, [&](auto tag) {
    return by_row_width(a.H, [&](auto tpr, auto ch) {
      typedef decltype(tag) Elem;
      constexpr int TPR = decltype(tpr)::value, CH = decltype(ch)::value;
      constexpr int BLOCK = row_block<TPR>(), R = BLOCK / TPR;
      // as many blocks as a CU holds by registers, over 256 CUs: one round, no tail
      const int64_t rows = (static_cast<int64_t>(a.T) + R - 1) / R;
      const int64_t blocks = 256 * std::max(1, 1024 / BLOCK);
      auto* kern = a.gate_kind == MOE_GATE_CHANNEL ? residual_fwd_kernel<Elem, TPR, CH, MOE_GATE_CHANNEL>
                   : a.gate_kind == MOE_GATE_TOKEN ? residual_fwd_kernel<Elem, TPR, CH, MOE_GATE_TOKEN>
                   : a.gate_kind == MOE_GATE_FULL  ? residual_fwd_kernel<Elem, TPR, CH, MOE_GATE_FULL>
                                                   : residual_fwd_kernel<Elem, TPR, CH, MOE_GATE_NONE>;
      hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(std::min(rows, blocks))),
                         dim3(BLOCK), 0, s, a);
      return hipGetLastError();
    });
  });
}

// Blocks of the backward, over 256 CUs: what a CU holds of the wider ones, and 512 threads a CU of
// the narrow ones, whose partials (a row a block) cost more than the rows in flight gain
// (16384 x 2048, both norms and a gate: 86.1 us with two blocks a CU, 96.3 with four).
int64_t residual_bwd_groups(int T, int H) {
  int64_t groups = 0;
  (void)by_row_width(H, [&](auto tpr, auto) {
    constexpr int BLOCK = row_block<decltype(tpr)::value>(), R = BLOCK / decltype(tpr)::value;
    groups = std::min<int64_t>((static_cast<int64_t>(T) + R - 1) / R,
                               256 * std::max(1, (BLOCK <= 256 ? 512 : 1024) / BLOCK));
    return hipSuccess;
  });
  return groups;
}

hipError_t launch_residual_bwd(int dtype, const ResidualBwdArgs& a, hipStream_t s,
                               KernelTimer* tm) {
  TimedScope ts(tm, MOE_K_RESIDUAL_NORM_BWD, s);
  return dtype == MOE_BF16 ? launch_residual_bwd_bf16(a, s)
         : dtype == MOE_F16 ? launch_residual_bwd_f16(a, s)
                            : launch_residual_bwd_f32(a, s);
}

}  // namespace moe
