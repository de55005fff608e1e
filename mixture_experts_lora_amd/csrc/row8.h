// Eight consecutive elements of a row, the unit that the residual and linear kernels load, round
// and store, and that one dropout counter covers.
#pragma once

#include "device_common.h"
#include "moe_lora.h"

namespace moe {

// Eight consecutive elements as they are stored: 16 bytes of a 16-bit type, 32 of float.
template <typename T> struct Row8;
template <> struct Row8<bf16_t> {
  uint4 a;
  __device__ void load(const bf16_t* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ void store(bf16_t* p) const { *reinterpret_cast<uint4*>(p) = a; }
  __device__ void zero() { a = make_uint4(0, 0, 0, 0); }
  __device__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ void set(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = static_cast<uint32_t>(f32_to_bf16(v[2 * i])) |
             (static_cast<uint32_t>(f32_to_bf16(v[2 * i + 1])) << 16);
    a = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <> struct Row8<f16_t> {
  uint4 a;
  __device__ void load(const f16_t* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ void store(f16_t* p) const { *reinterpret_cast<uint4*>(p) = a; }
  __device__ void zero() { a = make_uint4(0, 0, 0, 0); }
  __device__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = static_cast<float>(__builtin_bit_cast(f16_t, static_cast<uint16_t>(w[i])));
      v[2 * i + 1] =
          static_cast<float>(__builtin_bit_cast(f16_t, static_cast<uint16_t>(w[i] >> 16)));
    }
  }
  __device__ void set(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<f16_t>(v[2 * i]))) |
             (static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<f16_t>(v[2 * i + 1])))
              << 16);
    a = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <> struct Row8<float> {
  float4 a, b;
  __device__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
  __device__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  __device__ void set(const float (&v)[8]) {
    a = make_float4(v[0], v[1], v[2], v[3]);
    b = make_float4(v[4], v[5], v[6], v[7]);
  }
};

// Calls go with a value of the storage type of `dtype`.
template <typename F>
hipError_t by_type(int dtype, F&& go) {
  if (dtype == MOE_BF16) return go(bf16_t{});
  if (dtype == MOE_F16) return go(f16_t{});
  return go(float{});
}

}  // namespace moe
