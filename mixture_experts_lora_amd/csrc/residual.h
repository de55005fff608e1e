// What the residual operator's forward and backward kernels share: sums over a row, and the gate.
#pragma once

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
      // lane l takes wave l % W's sums; a butterfly over W lanes then gives every lane the total
      a = s[2 * (lane & (W - 1))];
      b = s[2 * (lane & (W - 1)) + 1];
      static_assert(W == 4 || W == 8 || W == 16, "steps below");
      a += dpp_f32<kDppSwap1>(a);
      b += dpp_f32<kDppSwap1>(b);
      a += dpp_f32<kDppSwap2>(a);
      b += dpp_f32<kDppSwap2>(b);
      if (W >= 8) {
        a += dpp_f32<kDppHalfMirror>(a);
        b += dpp_f32<kDppHalfMirror>(b);
      }
      if (W >= 16) {
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

}  // namespace moe
