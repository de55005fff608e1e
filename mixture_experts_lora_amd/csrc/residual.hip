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
#include "residual_fwd.h"

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
  return launch_residual_rows<false>(dtype, a, s);
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
