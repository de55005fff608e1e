// Counter-based dropout shared by the element-wise kernel, the residual kernels and the linear
// epilogue: whether an element is kept depends only on (seed, offset + site, element index), so
// a forward and its backward draw the same mask and no mask is ever stored.
//
// Generator: Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy as
// 1, 2, 3", SC 2011). Key = seed; counter = (element index / 8, offset + site), both 64 bits.
// One counter gives 128 bits, used as 16 for each of 8 consecutive elements: element i of the 8
// takes half i % 2 (low first) of word i / 2, and is kept when that number is >= t,
// t = round(65536 p). 16 bits rather than 32 halve the integer multiplies, the kernels' largest
// cost beside memory; the price is that P(drop) is t / 65536, off p by at most 2^-17. Kept
// elements are scaled by 1 / P(keep) of the rounded probability, so the mean is exact.
#pragma once

#include "device_common.h"
#include "launch.h"  // DropArgs

namespace moe {

struct DropKey {
  uint32_t k0, k1, o0, o1;
};

__device__ __forceinline__ DropKey drop_key(const DropArgs& d) {
  DropKey k{};
  if (d.thr) {
    const uint64_t seed = static_cast<uint64_t>(d.rng[0]);
    const uint64_t off = static_cast<uint64_t>(d.rng[1]) + d.site;
    k.k0 = static_cast<uint32_t>(seed);
    k.k1 = static_cast<uint32_t>(seed >> 32);
    k.o0 = static_cast<uint32_t>(off);
    k.o1 = static_cast<uint32_t>(off >> 32);
  }
  return k;
}

__device__ __forceinline__ uint4 philox(const DropKey& k, uint64_t ctr) {
  uint32_t x0 = static_cast<uint32_t>(ctr), x1 = static_cast<uint32_t>(ctr >> 32);
  uint32_t x2 = k.o0, x3 = k.o1, k0 = k.k0, k1 = k.k1;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = static_cast<uint64_t>(0xD2511F53u) * x0;
    const uint64_t b = static_cast<uint64_t>(0xCD9E8D57u) * x2;
    // three-operand exclusive or (v_bitop3_b32)
    x0 = __builtin_amdgcn_bitop3_b32(static_cast<uint32_t>(b >> 32), x1, k0, 0x96);
    x2 = __builtin_amdgcn_bitop3_b32(static_cast<uint32_t>(a >> 32), x3, k1, 0x96);
    x1 = static_cast<uint32_t>(b);
    x3 = static_cast<uint32_t>(a);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(x0, x1, x2, x3);
}

// The 128 bits of elements 8 ctr .. 8 ctr + 7; zeros, which keep all, without dropout.
__device__ __forceinline__ uint4 drop_words(const DropArgs& d, const DropKey& k, uint64_t ctr) {
  return d.thr ? philox(k, ctr) : make_uint4(0, 0, 0, 0);
}

// Whether element i (0..7) of the words is kept. (The high half is >= t where the word is >=
// t 2^16.) Callers select by it rather than multiply, so that a dropped infinity or NaN gives 0.
__device__ __forceinline__ bool kept(const DropArgs& d, const uint4& r, int i) {
  const uint32_t w = i < 2 ? r.x : i < 4 ? r.y : i < 6 ? r.z : r.w;
  return i & 1 ? w >= d.thr << 16 : (w & 0xffffu) >= d.thr;
}

__device__ __forceinline__ float drop(const DropArgs& d, const uint4& r, int i, float v) {
  return kept(d, r, i) ? v * d.scale : 0.f;
}

}  // namespace moe
