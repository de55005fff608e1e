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
// may be the same buffer: a thread reads its elements before it writes them.
template <typename Elem, bool VEC>
__global__ __launch_bounds__(256) void dropout_kernel(const Elem* src, Elem* dst, int64_t n,
                                                      DropArgs d) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, i = c * 8;
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

// Statistics of a row held as CH chunks of 8 elements: chunk i of a thread is chunk
// lane + i TPR of the row (chunks past the row are skipped).
template <typename Elem, int TPR, int CH>
__device__ __forceinline__ void row_stats(const Row8<Elem> (&r)[CH], int lane, int cpr, int kind,
                                          float inv_h, float eps, RowSum<TPR>& sum, float& mean,
                                          float& rstd) {
  mean = 0.f;
  if (kind == MOE_NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if (lane + i * TPR >= cpr) continue;
      float v[8];
      r[i].get(v);
#pragma unroll
      for (int j = 0; j < 8; ++j) s += v[j];
    }
    mean = sum(s, 0.f).x * inv_h;
  }
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    if (lane + i * TPR >= cpr) continue;
    float v[8];
    r[i].get(v);
#pragma unroll
    for (int j = 0; j < 8; ++j) q += (v[j] - mean) * (v[j] - mean);
  }
  rstd = 1.0f / sqrtf(sum(q, 0.f).x * inv_h + eps);
}

// (shift + w) u + b of one chunk; b may be null.
template <typename Elem>
__device__ __forceinline__ void affine(float (&u)[8], const Elem* w, const Elem* b, int col,
                                       float shift) {
  Row8<Elem> r;
  float f[8];
  r.load(w + col);
  r.get(f);
#pragma unroll
  for (int j = 0; j < 8; ++j) u[j] *= shift + f[j];
  if (b) {
    r.load(b + col);
    r.get(f);
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] += f[j];
  }
}

// ------------------------------------------------------------------ forward
// TPR threads a row, the row in CH chunks of 8 elements a thread. Reads h and y, writes h' and
// x' once; the norms' vectors come from cache. A thread reads all of its h and y before it writes
// anything, so h' may be h.
template <typename Elem, int TPR, int CH>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void residual_fwd_kernel(ResidualArgs p) {
  constexpr int BLOCK = TPR < 256 ? 256 : TPR;
  static_assert(TPR == kWave || TPR == BLOCK, "a row belongs to a wave or to a block");
  __shared__ float slots[2][2 * (TPR / kWave)];
  const int lane = row_lane<TPR>();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (BLOCK / TPR) + row_in_block<TPR>();
  if (row >= p.T) return;  // whole waves; a block that owns one row never leaves early
  RowSum<TPR> sum{slots, 0};
  const int cpr = p.H / 8;
  const int64_t base = row * p.H;
  const Elem* h = static_cast<const Elem*>(p.h);
  const Elem* y = static_cast<const Elem*>(p.y);
  Row8<Elem> rh[CH], ry[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = lane + i * TPR;
    rh[i].zero();
    ry[i].zero();
    if (c < cpr) {
      if (y) ry[i].load(y + base + 8 * c);
      if (h) rh[i].load(h + base + 8 * c);
    }
  }
  float4 st = make_float4(0.f, 0.f, 0.f, 0.f);
  if (y) {
    if (p.post != MOE_NORM_NONE)
      row_stats<Elem, TPR, CH>(ry, lane, cpr, p.post, p.inv_h, p.eps, sum, st.x, st.y);
    const DropKey key = drop_key(p.drop);
    const Elem* gate = static_cast<const Elem*>(p.gate);
    float g = 1.f;
    if (p.gate_kind == MOE_GATE_TOKEN) g = gate_value(to_f32<Elem>(gate[row]), p.gate_sigmoid);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = lane + i * TPR;
      if (c >= cpr) continue;
      float v[8], u[8];
      ry[i].get(v);
      if (p.post != MOE_NORM_NONE) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = (v[j] - st.x) * st.y;
        affine<Elem>(v, static_cast<const Elem*>(p.w_post), static_cast<const Elem*>(p.b_post),
                     8 * c, p.shift);
      }
      if (p.drop.thr) {
        const uint4 rnd = drop_words(p.drop, key, static_cast<uint64_t>(row * cpr + c));
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = drop(p.drop, rnd, j, v[j]);
      }
      if (p.gate_kind == MOE_GATE_CHANNEL || p.gate_kind == MOE_GATE_FULL) {
        Row8<Elem> rg;
        float f[8];
        rg.load(gate + (p.gate_kind == MOE_GATE_FULL ? base : 0) + 8 * c);
        rg.get(f);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= gate_value(f[j], p.gate_sigmoid);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= g;
      }
      rh[i].get(u);
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] += p.alpha * v[j];
      rh[i].set(u);
    }
  }
  if (p.h_out) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = lane + i * TPR;
      if (c < cpr) rh[i].store(static_cast<Elem*>(p.h_out) + base + 8 * c);
    }
  }
  if (p.pre != MOE_NORM_NONE) {
    row_stats<Elem, TPR, CH>(rh, lane, cpr, p.pre, p.inv_h, p.eps, sum, st.z, st.w);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = lane + i * TPR;
      if (c >= cpr) continue;
      float u[8];
      rh[i].get(u);
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] = (u[j] - st.z) * st.w;
      affine<Elem>(u, static_cast<const Elem*>(p.w_pre), static_cast<const Elem*>(p.b_pre), 8 * c,
                   p.shift);
      Row8<Elem> o;
      o.set(u);
      o.store(static_cast<Elem*>(p.x_out) + base + 8 * c);
    }
  }
  if (lane == 0 && p.stats) p.stats[row] = st;
}

// Threads a row and chunks a thread. Forward: a wave holds rows up to 2048 wide, wider ones take a
// block (16384 x 2048: 59.7 us by waves, 63.1 by blocks; 16384 x 4096: 128 and 110.5 us).
template <typename F>
hipError_t by_width_fwd(int H, F&& go) {
  using std::integral_constant;
  if (H <= 512) return go(integral_constant<int, 64>(), integral_constant<int, 1>());
  if (H <= 1024) return go(integral_constant<int, 64>(), integral_constant<int, 2>());
  if (H <= 2048) return go(integral_constant<int, 64>(), integral_constant<int, 4>());
  if (H <= 4096) return go(integral_constant<int, 256>(), integral_constant<int, 2>());
  if (H <= 8192) return go(integral_constant<int, 512>(), integral_constant<int, 2>());
  return go(integral_constant<int, 512>(), integral_constant<int, 4>());
}

}  // namespace

hipError_t launch_dropout(int dtype, int64_t n, const DropArgs& d, const void* src, void* dst,
                          hipStream_t s, KernelTimer* tm) {
  TimedScope ts(tm, MOE_K_DROPOUT, s);
  const bool vec = ((reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst)) & 15) == 0;
  const dim3 grid(static_cast<unsigned>(((n + 7) / 8 + 255) / 256));
  return by_type(dtype, [&](auto tag) {
    using Elem = decltype(tag);
    auto* kern = vec ? dropout_kernel<Elem, true> : dropout_kernel<Elem, false>;
    hipLaunchKernelGGL(kern, grid, dim3(256), 0, s, static_cast<const Elem*>(src),
                       static_cast<Elem*>(dst), n, d);
    return hipGetLastError();
  });
}

hipError_t launch_residual_fwd(int dtype, const ResidualArgs& a, hipStream_t s, KernelTimer* tm) {
  TimedScope ts(tm, MOE_K_RESIDUAL_NORM, s);
  return by_type(dtype, [&](auto tag) {
    return by_width_fwd(a.H, [&](auto tpr, auto ch) {
      constexpr int TPR = decltype(tpr)::value, BLOCK = TPR < 256 ? 256 : TPR, R = BLOCK / TPR;
      hipLaunchKernelGGL((residual_fwd_kernel<decltype(tag), TPR, decltype(ch)::value>),
                         dim3(static_cast<unsigned>((static_cast<int64_t>(a.T) + R - 1) / R)),
                         dim3(BLOCK), 0, s, a);
      return hipGetLastError();
    });
  });
}

// Blocks of the backward: 1024 threads a CU over 256 CUs keep enough rows in flight, and each
// block adds a row of partials.
int64_t residual_bwd_groups(int T, int H) {
  const int threads = H <= 512 ? 64 : H <= 2048 ? 256 : H <= 4096 ? 512 : 1024;
  const int rows = threads < 256 ? 256 / threads : 1;
  return std::min<int64_t>((static_cast<int64_t>(T) + rows - 1) / rows,
                           256 * 1024 / std::max(threads, 256));
}

hipError_t launch_residual_bwd(int dtype, const ResidualBwdArgs& a, hipStream_t s,
                               KernelTimer* tm) {
  TimedScope ts(tm, MOE_K_RESIDUAL_NORM_BWD, s);
  return dtype == MOE_BF16 ? launch_residual_bwd_bf16(a, s)
         : dtype == MOE_F16 ? launch_residual_bwd_f16(a, s)
                            : launch_residual_bwd_f32(a, s);
}

}  // namespace moe
