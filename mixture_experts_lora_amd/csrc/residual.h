// What the residual operator's forward and backward kernels share: sums over a row, and the gate.
#pragma once

#include <type_traits>

#include "device_common.h"
#include "launch.h"

namespace moe {

// ------------------------------------------------------------------ reductions over a row
// A row belongs to TPR threads: one wave, or a whole block of TPR / 64 waves that meets in LDS
// (one barrier a reduction: two slots in turn, so a wave that is one reduction ahead writes the
// slot that nobody reads any more). Every thread gets the same sum, in a fixed order.
template <int TPR>
struct RowSum {
  static constexpr int W = TPR / kWave;
  float (*slots)[2 * W];
  int turn;
  __device__ float2 operator()(float a, float b) {
    a = wave_sum(a);
    b = wave_sum(b);
    if constexpr (W == 1) {
      return make_float2(a, b);
    } else {
      float* s = slots[turn];
      turn ^= 1;
      const int wave = threadIdx.x / kWave, lane = threadIdx.x & (kWave - 1);
      if (lane == 0) {
        s[2 * wave] = a;
        s[2 * wave + 1] = b;
      }
      __syncthreads();
      // lane l takes wave l % P's sums (P: W's next power of two); a butterfly over P lanes then
      // gives every lane the total
      constexpr int P = W <= 2 ? 2 : W <= 4 ? 4 : W <= 8 ? 8 : 16;
      static_assert(W <= 16, "steps below");
      const int from = lane & (P - 1);
      a = from < W ? s[2 * from] : 0.f;
      b = from < W ? s[2 * from + 1] : 0.f;
      a += dpp_f32<kDppSwap1>(a);
      b += dpp_f32<kDppSwap1>(b);
      if (P >= 4) {
        a += dpp_f32<kDppSwap2>(a);
        b += dpp_f32<kDppSwap2>(b);
      }
      if (P >= 8) {
        a += dpp_f32<kDppHalfMirror>(a);
        b += dpp_f32<kDppHalfMirror>(b);
      }
      if (P >= 16) {
        a += dpp_f32<kDppMirror>(a);
        b += dpp_f32<kDppMirror>(b);
      }
      return make_float2(a, b);
    }
  }
};

// A thread's place in its row, and the row's place in its block, wave-uniform so that the row's
// addresses stay in scalar registers.
template <int TPR>
__device__ __forceinline__ int row_lane() {
  return TPR == kWave ? threadIdx.x & (kWave - 1) : threadIdx.x;
}
template <int TPR>
__device__ __forceinline__ int row_in_block() {
  return TPR == kWave ? __builtin_amdgcn_readfirstlane(threadIdx.x / kWave) : 0;
}

__device__ __forceinline__ float gate_value(float g, int sigmoid) {
  return sigmoid ? sigmoidf_(g) : g;
}
// The sigmoid and its slope s(g) (1 - s(g)) = s(g) s(-g) from t = exp(-|g|) alone: 1 / (1 + t) is the
// larger of s(g) and s(-g), t / (1 + t) the other. (1 - s would cancel for large g, down to 0 where s
// rounds to 1; two sigmoids cost a gate per element 4% of the backward.)
__device__ __forceinline__ float gate_slope(float g, float& value) {
  const float t = __expf(-fabsf(g)), r = __builtin_amdgcn_rcpf(1.f + t);
  value = g < 0.f ? t * r : r;
  return t * r * r;
}

// Threads of a block whose rows take TPR threads each: four rows of a wave, or one row.
template <int TPR>
constexpr int row_block() {
  return TPR == kWave ? 4 * kWave : TPR;
}

// Calls go with the threads a row takes and the chunks of 8 elements each of them takes: one chunk
// while a block can hold the row (registers decide how many rows are in flight). The widths leave
// lanes idle in between, most just above a step and in rows narrower than a wave's 512 elements
// (forward, bf16, one norm: 16384 x 1032 takes 34 us where a copy takes 27, 32768 x 64 takes 13.9 for
// a copy's 3.3). Rows above 8192 take two chunks a thread at 128 registers, which most variants pass:
// they spill (2048 x 16384 bf16, forward: 51 us with one norm, a copy's 53, but 82 with two norms, a
// gate and dropout; backward: 74 and 284 us where copies take 66 and 79).
template <typename F>
hipError_t by_row_width(int H, F&& go) {
  using std::integral_constant;
  using One = integral_constant<int, 1>;
  if (H <= 512) return go(integral_constant<int, 64>(), One());
  if (H <= 1024) return go(integral_constant<int, 128>(), One());
  if (H <= 2048) return go(integral_constant<int, 256>(), One());
  if (H <= 3584) return go(integral_constant<int, 448>(), One());
  if (H <= 4096) return go(integral_constant<int, 512>(), One());
  if (H <= 7168) return go(integral_constant<int, 896>(), One());
  if (H <= 8192) return go(integral_constant<int, 1024>(), One());
  return go(integral_constant<int, 1024>(), integral_constant<int, 2>());
}

}  // namespace moe
